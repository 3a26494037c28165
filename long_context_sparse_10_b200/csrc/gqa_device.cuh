// Device helpers shared by the grouped-head (GQA) kernels: waits of converged
// warps, TMEM loads without an own wait, two-wide fp32 arithmetic, and the page
// pool.
#pragma once

#include "common.cuh"
#include "tc.cuh"

namespace csa {
namespace gqa {

// D(TMEM) += A(TMEM, bf16 pairs) * B(shared)
__device__ __forceinline__ void mma_bf16_ts(uint32_t tmem_d, uint32_t tmem_a, uint64_t bdesc, uint32_t idesc,
                                            uint32_t accumulate) {
  asm volatile(
      "{\n.reg .pred p;\nsetp.ne.b32 p, %4, 0;\n"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(tmem_d),
      "r"(tmem_a), "l"(bdesc), "r"(idesc), "r"(accumulate));
}

// 32 columns without a wait; fence_regs() after the wait keeps uses behind it.
__device__ __forceinline__ void tmem_ld32_async(uint32_t taddr, float* v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]),
        "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]),
        "=f"(v[16]), "=f"(v[17]), "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]),
        "=f"(v[24]), "=f"(v[25]), "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, float* v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n"
      "tcgen05.wait::ld.sync.aligned;\n"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]),
        "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const float* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};\n" ::"r"(
          taddr),
      "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]), "f"(v[8]), "f"(v[9]),
      "f"(v[10]), "f"(v[11]), "f"(v[12]), "f"(v[13]), "f"(v[14]), "f"(v[15])
      : "memory");
}
__device__ __forceinline__ void fence_regs(float* v) {
#pragma unroll
  for (int i = 0; i < 32; i += 8)
    asm volatile("" : "+f"(v[i]), "+f"(v[i + 1]), "+f"(v[i + 2]), "+f"(v[i + 3]), "+f"(v[i + 4]), "+f"(v[i + 5]),
                      "+f"(v[i + 6]), "+f"(v[i + 7]));
}

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The same, kept in the source's order.
__device__ __forceinline__ float exp2_in_order(float x) {
  float y;
  asm volatile("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Two fp32 operations in one instruction (each rounded as its scalar form).
__device__ __forceinline__ void fma2(float& d0, float& d1, float a0, float a1, float b, float c) {
  asm("{\n.reg .b64 a, b, c, d;\nmov.b64 a, {%2, %3};\nmov.b64 b, {%4, %4};\nmov.b64 c, {%5, %5};\n"
      "fma.rn.f32x2 d, a, b, c;\nmov.b64 {%0, %1}, d;\n}\n"
      : "=f"(d0), "=f"(d1)
      : "f"(a0), "f"(a1), "f"(b), "f"(c));
}
// d = d * b + c, with c of each.
__device__ __forceinline__ void fma2v(float& d0, float& d1, float b, float c0, float c1) {
  asm("{\n.reg .b64 b, c, d;\nmov.b64 b, {%2, %2};\nmov.b64 c, {%3, %4};\nmov.b64 d, {%0, %1};\n"
      "fma.rn.f32x2 d, d, b, c;\nmov.b64 {%0, %1}, d;\n}\n"
      : "+f"(d0), "+f"(d1)
      : "f"(b), "f"(c0), "f"(c1));
}
__device__ __forceinline__ void add2(float& d0, float& d1, float a0, float a1) {
  asm("{\n.reg .b64 a, d;\nmov.b64 a, {%2, %3};\nmov.b64 d, {%0, %1};\nadd.rn.f32x2 d, d, a;\n"
      "mov.b64 {%0, %1}, d;\n}\n"
      : "+f"(d0), "+f"(d1)
      : "f"(a0), "f"(a1));
}

// (a0, a1) + (b, b) and (a0, a1) * (b0, b1) + (c, c), as above.
__device__ __forceinline__ void add2s(float& d0, float& d1, float a0, float a1, float b) {
  asm("{\n.reg .b64 a, b, d;\nmov.b64 a, {%2, %3};\nmov.b64 b, {%4, %4};\nadd.rn.f32x2 d, a, b;\n"
      "mov.b64 {%0, %1}, d;\n}\n"
      : "=f"(d0), "=f"(d1)
      : "f"(a0), "f"(a1), "f"(b));
}
__device__ __forceinline__ void sub2(float& d0, float& d1, float a0, float a1) {  // d - a
  asm("{\n.reg .b64 a, b, d;\nmov.b64 a, {%2, %3};\nmov.b64 b, {%4, %4};\nmov.b64 d, {%0, %1};\n"
      "fma.rn.f32x2 d, a, b, d;\nmov.b64 {%0, %1}, d;\n}\n"
      : "+f"(d0), "+f"(d1)
      : "f"(a0), "f"(a1), "f"(-1.f));
}
__device__ __forceinline__ void mul2(float& d0, float& d1, float a0, float a1, float b0, float b1) {
  asm("{\n.reg .b64 a, b, d;\nmov.b64 a, {%2, %3};\nmov.b64 b, {%4, %5};\nmul.rn.f32x2 d, a, b;\n"
      "mov.b64 {%0, %1}, d;\n}\n"
      : "=f"(d0), "=f"(d1)
      : "f"(a0), "f"(a1), "f"(b0), "f"(b1));
}
__device__ __forceinline__ void mul_add2(float& d0, float& d1, float b0, float b1, float c) {  // d * b + c
  asm("{\n.reg .b64 b, c, d;\nmov.b64 b, {%2, %3};\nmov.b64 c, {%4, %4};\nmov.b64 d, {%0, %1};\n"
      "fma.rn.f32x2 d, d, b, c;\nmov.b64 {%0, %1}, d;\n}\n"
      : "+f"(d0), "+f"(d1)
      : "f"(b0), "f"(b1), "f"(c));
}

// 2^x of two numbers on the fp32 units.  x = n + f with n the nearest whole
// number (adding 1.5 * 2^23 leaves it in the low bits of the sum) and |f| <= 1/2;
// 2^f by its minimax polynomial of degree 4 in relative error (fitted by
// iteratively reweighted least squares; 2.7e-6 off at most in fp32), and n is
// multiplied in as a power of two built from those low bits.  Below 2^-126 the
// result stays there; NaN stays NaN.
__device__ __forceinline__ void exp2_fma2(float& x0, float& x1) {
  constexpr float kMagic = 12582912.f;
  asm("max.NaN.f32 %0, %0, %1;" : "+f"(x0) : "f"(-126.f));
  asm("max.NaN.f32 %0, %0, %1;" : "+f"(x1) : "f"(-126.f));
  float t0, t1, n0, n1;
  add2s(t0, t1, x0, x1, kMagic);
  add2s(n0, n1, t0, t1, -kMagic);
  sub2(x0, x1, n0, n1);
  float y0, y1;
  fma2(y0, y1, x0, x1, 0.009570102207362652f, 0.05591785907745361f);
  mul_add2(y0, y1, x0, x1, 0.240247443318367f);
  mul_add2(y0, y1, x0, x1, 0.6931217908859253f);
  mul_add2(y0, y1, x0, x1, 0.9999992847442627f);
  mul2(x0, x1, y0, y1, __uint_as_float((__float_as_uint(t0) << 23) + 0x3f800000u),
       __uint_as_float((__float_as_uint(t1) << 23) + 0x3f800000u));
}

// Wait of a converged warp for a barrier's phase.  Almost always the phase is there or arrives within one try: that
// path has one try and a vote, so that no branch of it diverges (a loop whose exit is each lane's own costs 150
// clocks more).  The bounded loop is for the rest; false, for all lanes, when it runs out.
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, uint32_t limit = tc::kWaitLimit) {
  uint32_t ok;
  asm volatile(
      "{\n.reg .pred p;\nmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\nselp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  bool all = __all_sync(0xffffffffu, ok != 0);
  if (!all) all = __all_sync(0xffffffffu, tc::bar_wait_bounded(bar, parity, limit));
  return all;
}
// After a wait has run out: waits, with a limit, for the copies still in flight into a ring of `stages`, of which
// `loads` were issued.
__device__ __forceinline__ void await_copies(uint64_t* full, int stages, int loads) {
#pragma unroll 1
  for (int st = 0; st < stages && st < loads; ++st) wait_warp(&full[st], ((loads - 1 - st) / stages) & 1, 1u << 14);
}
// Arrives where `on` holds, without a branch.
__device__ __forceinline__ void bar_arrive_if(uint64_t* bar, bool on, uint32_t n = 1) {
  asm volatile("{\n.reg .pred p;\nsetp.ne.u32 p, %1, 0;\n@p mbarrier.arrive.shared::cta.b64 _, [%0], %2;\n}\n" ::"r"(
                   smem_u32(bar)),
               "r"(static_cast<uint32_t>(on)), "r"(n)
               : "memory");
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
// 32 bytes in one store where the address allows it: a warp whose lanes write 32 different rows pays per row.
__device__ __forceinline__ void st_global_32(void* p, const uint32_t* v, bool wide) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};\n" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]),
                 "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
  } else {
    reinterpret_cast<uint4*>(p)[0] = make_uint4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<uint4*>(p)[1] = make_uint4(v[4], v[5], v[6], v[7]);
  }
}
__device__ __forceinline__ void named_sync(int id, int threads) {
  asm volatile("bar.sync %0, %1;\n" ::"r"(id), "r"(threads) : "memory");
}

// Fetches a tensor map (a kernel parameter) ahead of its first use.
__device__ __forceinline__ void prefetch_map(const void* map) {
  asm volatile("prefetch.tensormap [%0];\n" ::"l"(map) : "memory");
}

// One lane of a converged warp (always the same one).
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n.reg .pred p;\nelect.sync _|p, 0xffffffff;\nselp.b32 %0, 1, 0, p;\n}\n" : "=r"(r));
  return r != 0;
}

// A pool of pages and one table of them.
struct Pool {
  uint4* k;  // 16-byte pieces
  uint4* v;
  float* mass;
  int64_t n_pages;
  int Hkv, page, kp, vp;  // kp, vp: pieces per token of k and v
  int shift;              // page = 1 << shift
};

// Slot (row of the pool's planes) of a position, or -1 where the table holds no page of the pool for it.
__device__ __forceinline__ int64_t slot_of(const Pool& c, const int32_t* table, int max_pages, int h, int pos) {
  const int pg = pos >> c.shift;
  if (pos < 0 || pg >= max_pages) return -1;
  const int id = __ldg(table + pg);
  if (id < 0 || id >= c.n_pages || !CSA_INBOUNDS(h >= 0 && h < c.Hkv)) return -1;
  return ((static_cast<int64_t>(id) * c.Hkv + h) << c.shift) + (pos & (c.page - 1));
}

inline Pool pool_of(const gqa_cache* c) {
  Pool p;
  p.k = static_cast<uint4*>(c->k);
  p.v = static_cast<uint4*>(c->v);
  p.mass = c->mass;
  p.n_pages = c->n_pages;
  p.Hkv = c->n_kv_heads;
  p.page = c->page_size;
  p.shift = c->page_size == 16 ? 4 : (c->page_size == 32 ? 5 : (c->page_size == 64 ? 6 : 7));
  p.kp = c->d_qk / 8;
  p.vp = c->d_v / 8;
  return p;
}

}  // namespace gqa
}  // namespace csa

// Pairs of fp32: one instruction for both (each rounded to nearest by itself).
#pragma once

namespace ft {

namespace {

typedef unsigned long long Pair;

__device__ __forceinline__ Pair pair(float lo, float hi) {
    Pair p;
    asm("mov.b64 %0, {%1, %2};" : "=l"(p) : "f"(lo), "f"(hi));
    return p;
}
__device__ __forceinline__ float2 halves(Pair p) {
    float2 f;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(p));
    return f;
}
__device__ __forceinline__ Pair add2(Pair a, Pair b) {
    Pair d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ Pair mul2(Pair a, Pair b) {
    Pair d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ Pair fma2(Pair a, Pair b, Pair c) {
    Pair d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
// b - a
__device__ __forceinline__ Pair from2(Pair a, Pair b) { return fma2(a, pair(-1.f, -1.f), b); }
__device__ __forceinline__ Pair neg2(Pair a) { return a ^ 0x8000000080000000ULL; }
__device__ __forceinline__ Pair swap2(Pair a) {
    const float2 f = halves(a);
    return pair(f.y, f.x);
}

}  // namespace

}  // namespace ft

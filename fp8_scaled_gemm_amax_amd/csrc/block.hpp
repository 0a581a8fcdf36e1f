// block.hpp - host-side launchers of the gated feed-forward product and of the
// adapters, internal to the library as kernels.hpp; arguments were validated by
// the C ABI layer.
#pragma once

#include "kernels.hpp"

namespace fp8amax {

// The gated product: h = a b^T with b's gate rows 0 .. inter-1 and up rows inter ..
// 2 inter-1, act = silu(h gate) * h up; h NULL: not stored.
struct GluFwd {
    const uint8_t* a;
    int64_t lda;
    const uint8_t* b;
    int64_t ldb;
    int64_t m, inter, k;
    const float* sa;
    int sa_vec;
    const float* sb;
    int sb_vec;
    uint16_t* act;
    int64_t ldact;
    uint16_t* h;
    int64_t ldh;
};

// Its backward pass: da = a b^T [m x inter], dh = SwiGLU's gradient at h; act
// (NULL: not stored) from the same read of h.
struct GluBwd {
    const uint8_t* a;
    int64_t lda;
    const uint8_t* b;
    int64_t ldb;
    int64_t m, inter, k;
    const float* sa;
    int sa_vec;
    const float* sb;
    int sb_vec;
    const uint16_t* h;
    int64_t ldh;
    uint16_t* dh;
    int64_t lddh;
    uint16_t* act;
    int64_t ldact;
};

hipError_t launch_gemm_swiglu(const GluFwd& p, int fa, int fb, hipStream_t st);
hipError_t launch_gemm_swiglu_backward(const GluBwd& p, int fa, int fb, hipStream_t st);

// Adapters: out = base + scaling_e (x A_e^T) B_e^T, e = adapter[token], in two
// launches; ws holds the sums of x A^T over parts of k.
constexpr int kLoraMaxRank = 128;
constexpr int kLoraMaxParts = 16;               // parts of k
constexpr int64_t kLoraPartRows = 8192;         // parts * tokens, unless one part each is more

struct Lora {
    const uint16_t* x;
    int64_t tokens, k, ldx;
    const int32_t* adapter;
    int adapters, rank;
    const uint16_t* a;                          // [adapters x rank x k]
    int64_t lda, gsa;
    const uint16_t* b;                          // [adapters x n x rank]
    int64_t ldb, gsb;
    const float* scaling;
    int64_t n;
    const uint16_t* base;                       // NULL: zeros
    int64_t ldbase;
    uint16_t* out;
    int64_t ldout;
    float* ws;
    int parts;                                  // the launcher's
};

// Rows of partial sums that a call of these sizes may use.
inline int64_t lora_part_rows(int64_t tokens) {
    const int64_t most = kLoraMaxParts * tokens < kLoraPartRows ? kLoraMaxParts * tokens : kLoraPartRows;
    return tokens > most ? tokens : most;
}

hipError_t launch_lora_add(const Lora& p, hipStream_t st);

}  // namespace fp8amax

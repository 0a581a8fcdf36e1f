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

// Whether the kernel for a few rows takes a call of m rows (else tiles of 64 rows do). Up to
// 16 rows it does; with 17 to 32 its loads of a's rows weigh as much as the weights, and tiles
// of 64 x 64 outputs are faster where they occupy a good part of the CUs once. Few rows' kernel
// and tiles (32 rows, us on the device): 2048 x 1408 6.1 and 9.4, 4096 x 4096 (64 tiles) 11.0
// and 14.2, x 6144 (96) 15.8 and 14.2, x 11008 (172) 24 and 18.6, x 14336 (224) 31.8 and 29.7,
// 8192 x 28672 (448, so a second round of tiles) 91 and 94; 17 rows 5.6 and 9.7, 11.0 and 14.2,
// 13.8 and 14.4, 24.2 and 18.3, 30.0 and 29.7, 83 and 94; 33 rows of 4096 x 14336 42 and 30.
constexpr int kFewRows = 32;
inline bool glu_few_rows(int64_t m, int64_t inter, int64_t cus) {
    const int64_t tiles = (inter + 63) / 64;
    return m <= 16 || (m <= kFewRows && (tiles * 8 < cus * 3 || tiles > cus));
}

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

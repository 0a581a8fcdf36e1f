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
// 13.8 and 14.4, 24.2 and 18.3, 30.0 and 29.7, 83 and 94; 16 rows 4.9 and 9.0, 10.3 and 14.0,
// 12.6 and 14.0, 19.4 and 17.7, 29.3 and 29.1, 75 and 92; 33 rows of 4096 x 14336 42 and 30.
constexpr int kFewRows = 32;
inline bool glu_few_rows(int64_t m, int64_t inter, int64_t cus) {
    const int64_t tiles = (inter + 63) / 64;
    return m <= 16 || (m <= kFewRows && (tiles * 8 < cus * 3 || tiles > cus));
}

// Large tiles where those of a quarter of their size would take a CU more than one.
// On 256 CUs: product of 512 x 4096 x 7168 (112 large tiles) 41 us, 45 in 128 x 128 tiles; of
// 256 x 4096 x 8192 (64) 41 and 24; gradient of 2048 x 4096 x 4096 (128) 50 and 58, of
// 1024 x 4096 x 4096 (64) 46 and 29.
inline bool glu_large_tiles(int64_t large, int64_t cus) { return large * 4 > cus; }

// Tiles of 64 rows where those of 128 would leave half of the CUs idle, or half of
// each tile empty. On 256 CUs, with them and without: product of 300 x 2048 x 1408 10.2 and
// 13.7 us, 64 x 4096 x 14336 30 and 32, gradient of 1001 x 2048 x 1408 13.5 and 19.2. Past the
// limit: product of 777 x 2048 x 1408 (154 tiles of 128) 18.8 and 14.9, gradient of
// 200 x 4096 x 14336 (224) 35 and 29.
inline bool glu_tiles_of_64_rows(int64_t m, int64_t tiles128, int64_t cus) { return m <= 64 || tiles128 * 2 <= cus; }

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

// Block-scaled FP8 product on tiles:
//   Y[m,n] = sum_b SCA[b,m] SCB[n/128,b] / 448^2 * (sum_{k in block b} CA[m,k] CB[n,k]),
// as a dense product (+ bias, 16-bit Y), and over rows grouped by expert for
// the two products of a mixture's feed-forward block:
//   kGateUp  rows gathered from the tokens' codes, weight rows n and I + n
//            (gate and up) side by side in one tile; h = silu(g) * u leaves
//            the tile as E4M3 codes with one scale per 128 channels;
//   kDown    h's codes against the down weights; rows out as 16-bit integers with
//            one scale per 128 channels (a later kernel weights and sums a
//            token's rows).  fp32 rows would be twice the bytes, the largest
//            share of the prefill's traffic; the integers are within 2^-16 of a
//            block's largest value, below the rounding of a 16-bit Y.
//
// One v_mfma_f32_16x16x128_f8f6f4 covers a whole scale block of K, from a zero
// accumulator; its 16 x 16 result is then added into fp32 registers times the
// block's scale, SCA * SCB, by ordinary fused multiply-adds.  The weight is
// the MFMA's first operand, so that a lane's four results belong to one token
// row (one scale) and four consecutive channels.
//
// A tile's K stages are 128 bytes of every row, in a ring of two LDS buffers
// filled by buffer loads that go straight to LDS; 16-byte chunk c of row r
// sits in slot c ^ ((r / 2) % 8), so 16 rows' fragment reads cover the banks
// evenly.  Stage kt + 1 loads while stage kt is multiplied.
#include "common.h"

namespace llmint8 {

namespace {

constexpr int kStageK = kBlock;  // bytes of K per stage: one scale block
constexpr int kMaxKb = (LLMINT8_K_MAX + kBlock - 1) / kBlock;
constexpr float kCodeScale = 1.0f / (448.0f * 448.0f);
constexpr int64_t kMaxGrid = 0x7fffff;  // workgroups of up to 512 threads: below 2^32 threads
constexpr uint32_t kPastEnd = 0xffffff00u;  // a buffer offset that reads 0

enum BlockMode { kDense, kGateUp, kDown };

__device__ __forceinline__ v4f mfma_block(const v8i& w, const v8i& x) {
    const v4f zero = {0.0f, 0.0f, 0.0f, 0.0f};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, x, zero, 0, 0, 0, 0, 0, 0);
}

// lane p's 4 bytes at base + off land in LDS at lds_addr + 4 p
__device__ __forceinline__ void dma4(const float* base, uint32_t off, uint32_t lds_addr) {
    uint32_t saved;
    asm volatile(
        "s_mov_b32 %0, m0\n\t"
        "s_mov_b32 m0, %1\n\t"
        "s_nop 0\n\t"
        "global_load_lds_dword %2, %3\n\t"
        "s_mov_b32 m0, %0"
        : "=&s"(saved)
        : "s"(lds_addr), "v"(off), "s"(base)
        : "memory");
}

// Workgroups go round-robin over the 8 XCDs: block b of `total` becomes place
// L of an order in which each XCD walks a contiguous range.
__device__ __forceinline__ int xcd_order(int b, int total) {
    const int q = total >> 3, r = total & 7, x = b & 7;
    return x * q + min(x, r) + (b >> 3);
}

// A workgroup's waves stand WM x WN on its tile; every wave has NT = 4 channel
// tiles of 16 and up to kMaxMT row tiles of 16.
template <int WM_, int WN_, int kMaxMT_>
struct Shape {
    static constexpr int WM = WM_, WN = WN_, NW = WM * WN, kMaxMT = kMaxMT_;
    static constexpr int BM = 16 * WM * kMaxMT, BN = 256, NT = BN / WN / 16;
    static constexpr int kStageBytes = (BM + BN) * kStageK;
    static constexpr int kSa = BM < 64 ? 64 : BM;  // floats of a stage's row scales
    static_assert(NT == 4 && WN == 4, "a wave's 64 channels: half a weight block, or gate and up of 32");
};

struct Tile {
    int row0, rows, n0, e;  // rows [row0, row0 + rows), channels from n0 of weight matrix e
};

// The tile's work with MT row tiles per wave (rows <= 16 WM MT).
template <typename S, int MODE, bool BF16, int MT>
__device__ __forceinline__ void tile_body(const BlockGemmArgs& a, const Tile& tile, int8_t* ring, float* s_sa,
                                          float* s_sb) {
    constexpr int BM = 16 * S::WM * MT, BN = S::BN, NT = S::NT;
    constexpr int kDmaA = BM / 8 / S::NW, kDmaB = BN / 8 / S::NW;  // 8-row loads per wave and stage
    static_assert(kDmaB * 8 * S::NW == BN && kDmaA * 8 * S::NW == BM, "whole loads per wave");
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / S::WN, wn = wave % S::WN;
    const int K = a.K, nkb = (K + kBlock - 1) / kBlock;
    const int row0 = tile.row0, rows = tile.rows, n0 = tile.n0, e = tile.e;

    // ---- stage loads: one instruction = 8 rows x 128 bytes; lane p fills slot
    // p % 8 of row p / 8 and so fetches logical chunk (p % 8) ^ ((row / 2) % 8).
    // Rows past the descriptor's read 0 (their results are never stored).
    const uint8_t* base_a = a.CA;
    const uint8_t* base_b;
    uint32_t bytes_a, bytes_b;
    if constexpr (MODE == kGateUp) {
        bytes_a = (uint32_t)((int64_t)a.M * K);  // gathered rows (below 2^32 bytes in all)
        base_b = a.CB + (size_t)e * 2 * a.N * K;
        bytes_b = (uint32_t)((int64_t)2 * a.N * K);
    } else {
        base_a += (size_t)row0 * K;
        bytes_a = (uint32_t)rows * (uint32_t)K;
        base_b = a.CB + ((size_t)e * a.N + n0) * K;
        bytes_b = (uint32_t)min(BN, a.N - n0) * (uint32_t)K;
    }
    const v4i rsrc_a = buffer_rsrc(base_a, bytes_a), rsrc_b = buffer_rsrc(base_b, bytes_b);
    // byte of the row where this lane's chunk starts, in even groups of 8 rows;
    // odd groups flip bit 6
    const uint32_t ch = ((lane & 7) ^ (lane >> 4)) * 16;
    // rows of a wave's loads: A rows 8 kDmaA wave + 8 d + lane / 8 of the tile
    // (kGateUp: of the tokens the tile's rows come from), B rows likewise; in
    // kGateUp a consumer wave's 64 rows are the gates of its 32 channels, then
    // the ups (channels past N read some other row: their h is set to 0)
    uint32_t row_a[MODE == kGateUp ? kDmaA : 1];
    if constexpr (MODE == kGateUp) {
#pragma unroll
        for (int d = 0; d < kDmaA; ++d) {
            const int r = min(8 * (kDmaA * wave + d) + (lane >> 3), rows - 1);
            row_a[d] = (uint32_t)a.row_token[row0 + r] * (uint32_t)K;
        }
    } else {
        row_a[0] = (uint32_t)(8 * kDmaA * wave + (lane >> 3)) * (uint32_t)K;
    }
    uint32_t row_b = (uint32_t)(lane >> 3);
    if constexpr (MODE == kGateUp) {
        const int r = 8 * kDmaB * wave;  // (a multiple of 32: whole halves)
        static_assert(MODE != kGateUp || 8 * kDmaB % 32 == 0, "loads of a wave stay in one half");
        row_b += (uint32_t)(n0 + (r >> 6) * 32);
        row_b += (uint32_t)(((r >> 5) & 1) * a.N);
    } else {
        row_b += (uint32_t)(8 * kDmaB * wave);
    }
    row_b *= (uint32_t)K;
    // the row scales: lane p of each instruction one row of 64
    uint32_t sa_off;
    {
        const int r = min((64 * wave + lane) % S::kSa, rows - 1);
        sa_off = 4 * (uint32_t)(MODE == kGateUp ? a.row_token[row0 + r] : r);
    }
    const float* sa_base = MODE == kGateUp ? a.SCA : a.SCA + row0;
    const uint32_t lds_ring = __builtin_amdgcn_readfirstlane(lds_address(ring));
    const uint32_t lds_sa = __builtin_amdgcn_readfirstlane(lds_address(reinterpret_cast<const int8_t*>(s_sa)));
    const int half_kt = K % kStageK != 0 ? nkb - 1 : -1;  // the stage whose second half is past K
    // load d of a wave's kDma per stage: A rows, B rows, the row scales.  Past
    // the last stage it re-reads that one, into a buffer nobody reads again.
    constexpr int kDma = kDmaA + kDmaB + 1;
    static_assert(kDmaB % 2 == 0, "parity of the 8-row groups");
    auto dma = [&](int d, int kt_want, int u) {
        const int kt = min(kt_want, nkb - 1);
        const uint32_t kd = (uint32_t)kt * kStageK;
        if (d < kDmaA) {
            const int grp = kDmaA * wave + d;
            const uint32_t c = ch ^ ((uint32_t)((kDmaA % 2 == 0 ? d : wave + d) & 1) << 6);
            const uint32_t row = MODE == kGateUp ? row_a[MODE == kGateUp ? d : 0] + kd
                                                 : row_a[0] + (kd + (uint32_t)(8 * d) * (uint32_t)K);
            dma_line(rsrc_a, kt == half_kt && c >= 64 ? kPastEnd : row + c, lds_ring + u * S::kStageBytes + grp * 8 * kStageK);
        } else if (d < kDmaA + kDmaB) {
            const int i = d - kDmaA, grp = kDmaB * wave + i;
            const uint32_t c = ch ^ ((uint32_t)(i & 1) << 6);
            uint32_t step = (uint32_t)(8 * i);
            if (MODE == kGateUp && i >= 4) step += (uint32_t)(a.N - 32);  // (a wave of 64 rows: its up half)
            dma_line(rsrc_b, kt == half_kt && c >= 64 ? kPastEnd : row_b + (kd + step * (uint32_t)K) + c,
                     lds_ring + u * S::kStageBytes + (S::BM + grp * 8) * kStageK);
        } else {
            dma4(sa_base + (int64_t)kt * a.ld_sa, sa_off, lds_sa + (u * S::kSa + 64 * wave % S::kSa) * 4);
        }
    };

    // ---- fragments: lane l holds 32 bytes of row (l % 16), chunks l / 16 and
    // l / 16 + 4 (the same K order for both operands).  The addresses of the
    // wave's first rows in the current buffer; `other` leads to the other one.
    constexpr int kWaveM = MT * 16, kWaveN = NT * 16;
    const int fr = lane & 15;
    const uint32_t f_lo = fr * kStageK + (((lane >> 4) ^ (fr >> 1)) & 7) * 16;
    uint32_t at_x[2] = {lds_ring + wm * kWaveM * kStageK + f_lo, lds_ring + wm * kWaveM * kStageK + (f_lo ^ 64)};
    uint32_t at_w[2] = {at_x[0] + (S::BM + wn * kWaveN - wm * kWaveM) * kStageK,
                        at_x[1] + (S::BM + wn * kWaveN - wm * kWaveM) * kStageK};
    uint32_t at_sa = lds_sa + (wm * kWaveM + fr) * 4;
    int other = 1;
    auto flip = [&]() {
        at_x[0] += other * S::kStageBytes;
        at_x[1] += other * S::kStageBytes;
        at_w[0] += other * S::kStageBytes;
        at_w[1] += other * S::kStageBytes;
        at_sa += other * S::kSa * 4;
        other = -other;
    };
    auto frag = [&](const uint32_t (&at)[2], int row) -> v8i {
        const v4i lo = lds_at<v4i>(at[0] + row * kStageK), hi = lds_at<v4i>(at[1] + row * kStageK);
        return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    };

    v4f acc[NT][MT];
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int j = 0; j < MT; ++j) acc[i][j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    // which half's weight scale a wave's channel tiles take
    const float* sb_at = s_sb + (MODE == kGateUp ? 0 : wn * kWaveN / kBlock) * kMaxKb;

    // The K loop.  Row tile j's MFMAs fill p[j % 2] while the results of the
    // row tile before are scaled and added; its activations are read one row
    // tile ahead.  Between the stage's last two row tiles every wave waits for
    // its loads of the next stage and its reads of this one, and meets the
    // others: the next stage is in the other buffer, this one is free.  The last
    // row tile reads the next stage's weights in place, and the loads of the
    // stage after go out with it and with the first row tile that follows.
    static_assert(MT % 2 == 0, "the row tiles alternate between two register sets");
    v8i w[NT], x[2];
    v4f p[2][NT];
    float sa[2], sb0, sb1;
    float f0 = 0.0f, f1 = 0.0f;  // scales of the results in flight (gate or all, up)
    auto read_sa = [&](int j) { return lds_at<float>(at_sa + 64 * j); };
    auto read_sb = [&](int kt) {
        sb0 = sb_at[kt];
        sb1 = MODE == kGateUp ? sb_at[kMaxKb + kt] : sb0;
    };
    auto add = [&](int i, int j, int set) {
        const float f = MODE == kGateUp && i >= NT / 2 ? f1 : f0;
#pragma unroll
        for (int v = 0; v < 4; ++v) acc[i][j][v] = __builtin_fmaf(p[set][i][v], f, acc[i][j][v]);
    };
#pragma unroll
    for (int i = 0; i < NT; ++i) p[1][i] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    auto stage = [&](int kt) {
        const int u = kt & 1;
#pragma unroll
        for (int j = 0; j < MT; ++j) {
            if (j == MT - 1) {
                __builtin_amdgcn_s_waitcnt(0);
                stage_barrier();
                flip();
                x[0] = frag(at_x, 0);  // (x[0]'s last use has been issued)
                sa[0] = read_sa(0);
            } else {
                x[(j + 1) & 1] = frag(at_x, 16 * (j + 1));
                sa[(j + 1) & 1] = read_sa(j + 1);
            }
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                p[j & 1][i] = mfma_block(w[i], x[j & 1]);
                if (j == MT - 1) w[i] = frag(at_w, 16 * i);
                add(i, (j + MT - 1) % MT, (j + 1) & 1);
                if (j == MT - 1)
#pragma unroll
                    for (int d = i * (kDma / 2) / NT; d < (i + 1) * (kDma / 2) / NT; ++d) dma(d, kt + 2, u);
                if (j == 0)
#pragma unroll
                    for (int d = kDma / 2 + i * (kDma - kDma / 2) / NT;
                         d < kDma / 2 + (i + 1) * (kDma - kDma / 2) / NT; ++d)
                        dma(d, kt + 1, 1 - u);
                __builtin_amdgcn_sched_barrier(0);
            }
            f0 = sa[j & 1] * sb0;
            f1 = MODE == kGateUp ? sa[j & 1] * sb1 : f0;
            if (j == MT - 1) read_sb(min(kt + 1, nkb - 1));
        }
    };
    // stage 0 whole, and the part of stage 1 that the last row tile of a stage
    // before it would have loaded
#pragma unroll
    for (int d = 0; d < kDma; ++d) dma(d, 0, 0);
    // meanwhile the weight block scales of the tile's two 128-channel halves (gate
    // and up, or channels n0.. and n0 + 128..), with the codes' 1/448^2
    {
        const int nnb = (a.N + kBlock - 1) / kBlock;
        const float* sb_lo = a.SCB + ((size_t)e * (MODE == kGateUp ? 2 : 1) * nnb + n0 / kBlock) * nkb;
        const float* sb_hi = MODE == kGateUp ? sb_lo + (size_t)nnb * nkb : n0 + kBlock < a.N ? sb_lo + nkb : sb_lo;
        for (int i = tid; i < nkb; i += 64 * S::NW) {
            s_sb[i] = sb_lo[i] * kCodeScale;
            s_sb[kMaxKb + i] = sb_hi[i] * kCodeScale;
        }
    }
    __builtin_amdgcn_s_waitcnt(0);
    stage_barrier();
#pragma unroll
    for (int d = 0; d < kDma / 2; ++d) dma(d, 1, 1);
#pragma unroll
    for (int i = 0; i < NT; ++i) w[i] = frag(at_w, 16 * i);
    x[0] = frag(at_x, 0);
    sa[0] = read_sa(0);
    read_sb(0);
    for (int kt = 0; kt < nkb; ++kt) stage(kt);
#pragma unroll
    for (int i = 0; i < NT; ++i) add(i, MT - 1, (MT - 1) & 1);
    wait_vmcnt<0>();  // the loads past the last stage have landed too

    // ---- results: lane l holds channels 4 (l / 16) .. + 3 of each 16-channel
    // tile for token row l % 16 of each 16-row tile.  They leave through LDS (the
    // ring, free now) as whole 16-byte pieces of rows.
    const int cq = (lane >> 4) * 4;
    __syncthreads();  // every wave's loads and reads of the ring are done
    if constexpr (MODE != kGateUp) {
        // 16-bit values of the wave's 64 channels, 128 bytes per row: piece c of row
        // r in slot c ^ ((r / 2) % 8)
        int8_t* stage = ring + wave * kWaveM * 128;
        auto put = [&](int i, int j, const uint16_t (&y)[4]) {
            const int piece = (2 * i + (lane >> 5)) ^ (fr >> 1);
            *reinterpret_cast<uint2*>(stage + (16 * j + fr) * 128 + piece * 16 + ((lane >> 4) & 1) * 8) =
                make_uint2(y[0] | (uint32_t)y[1] << 16, y[2] | (uint32_t)y[3] << 16);
        };
        const int n_wave = n0 + wn * kWaveN;
        if constexpr (MODE == kDense) {
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                float b[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                if (a.bias != nullptr)
#pragma unroll
                    for (int v = 0; v < 4; ++v)
                        if (n_wave + 16 * i + cq + v < a.N) b[v] = widen16<BF16>(a.bias[n_wave + 16 * i + cq + v]);
#pragma unroll
                for (int j = 0; j < MT; ++j) {
                    uint16_t y[4];
#pragma unroll
                    for (int v = 0; v < 4; ++v) y[v] = narrow16<BF16>(acc[i][j][v] + b[v]);
                    put(i, j, y);
                }
            }
        } else {
            // a row's 128 channels (two waves) as 16-bit integers of their largest
            float* red = s_sb;  // [WN][BM], past its use
            static_assert(S::WN * S::BM <= 2 * kMaxKb, "room for the maxima");
#pragma unroll
            for (int j = 0; j < MT; ++j) {
                float m = 0.0f;
#pragma unroll
                for (int i = 0; i < NT; ++i)
#pragma unroll
                    for (int v = 0; v < 4; ++v) m = fmaxf(m, fabsf(acc[i][j][v]));
                m = fmaxf(m, __shfl_xor(m, 16));
                m = fmaxf(m, __shfl_xor(m, 32));
                if (lane < 16) red[wn * BM + wm * kWaveM + 16 * j + lane] = m;
            }
            __syncthreads();
#pragma unroll
            for (int j = 0; j < MT; ++j) {
                const int r = wm * kWaveM + 16 * j + fr;
                const float m = fmaxf(red[(wn & 2) * BM + r], red[((wn & 2) + 1) * BM + r]);
                const float f = m == 0.0f ? 0.0f : fminf(kPartMax / m, 3.402823466e38f);
                if ((wn & 1) == 0 && lane < 16 && r < rows && n_wave < a.N)
                    a.part_scale[(int64_t)(n_wave / kBlock) * a.ld_part + row0 + r] = m * (1.0f / kPartMax);
#pragma unroll
                for (int i = 0; i < NT; ++i) {
                    uint16_t y[4];
#pragma unroll
                    for (int v = 0; v < 4; ++v) y[v] = (uint16_t)(int16_t)__builtin_rintf(acc[i][j][v] * f);
                    put(i, j, y);
                }
            }
        }
        wave_fence();
        uint16_t* Y = (MODE == kDense ? a.Y : a.part) + (size_t)(row0 + wm * kWaveM) * a.N + n_wave;
        const int piece = lane & 7;
#pragma unroll
        for (int it = 0; it < 2 * MT; ++it) {
            const int r = 8 * it + (lane >> 3);
            if (wm * kWaveM + r >= rows) continue;
            const v4i y = *reinterpret_cast<const v4i*>(stage + r * 128 + (piece ^ ((r >> 1) & 7)) * 16);
            uint16_t* out = Y + (size_t)r * a.N + 8 * piece;
            if ((a.N & 7) == 0) {
                // non-temporal: written once, past the caches that hold the operands
                // (4096 x 28672 x 8192 794 -> 788 us)
                if (n_wave + 8 * piece < a.N) __builtin_nontemporal_store(y, reinterpret_cast<v4i*>(out));
            } else {
#pragma unroll
                for (int v = 0; v < 8; ++v)
                    if (n_wave + 8 * piece + v < a.N) out[v] = (uint16_t)((uint32_t)y[v >> 1] >> (16 * (v & 1)));
            }
        }
    } else {
        // h of 32 channels per wave; a row's maximum over the tile's 128
        // channels from the four waves that share its rows
        float* red = s_sb;  // [WN][BM], past its use
        int8_t* stage = ring;  // [BM] rows of 128 codes
#pragma unroll
        for (int j = 0; j < MT; ++j) {
            float m = 0.0f;
#pragma unroll
            for (int i = 0; i < NT / 2; ++i) {
                const bool in = n0 + wn * 32 + 16 * i + cq < a.N;
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                    const float h = in ? silu(acc[i][j][v]) * acc[i + NT / 2][j][v] : 0.0f;
                    acc[i][j][v] = h;
                    m = fmaxf(m, fabsf(h));
                }
            }
            m = fmaxf(m, __shfl_xor(m, 16));
            m = fmaxf(m, __shfl_xor(m, 32));
            if (lane < 16) red[wn * BM + wm * kWaveM + 16 * j + lane] = m;
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < MT; ++j) {
            const int r = wm * kWaveM + 16 * j + fr;
            const float m = fmaxf(fmaxf(red[r], red[BM + r]), fmaxf(red[2 * BM + r], red[3 * BM + r]));
            const float f = block_factor(m);
            if (wn == 0 && lane < 16 && r < rows) a.SH[(int64_t)(n0 / kBlock) * a.ld_sh + row0 + r] = m;
#pragma unroll
            for (int i = 0; i < NT / 2; ++i)
                *reinterpret_cast<uint32_t*>(stage + r * 128 + ((2 * wn + i) ^ (fr >> 1)) * 16 + cq) =
                    e4m3_pack4(acc[i][j][0], acc[i][j][1], acc[i][j][2], acc[i][j][3], f);
        }
        __syncthreads();
        uint8_t* H = a.H + (size_t)row0 * a.N + n0;
        for (int o = tid; o < BM * 8; o += 64 * S::NW) {
            const int r = o >> 3, piece = o & 7;
            if (r < rows && n0 + 16 * piece < a.N)  // (N is a multiple of 64)
                *reinterpret_cast<v4i*>(H + (size_t)r * a.N + 16 * piece) =
                    *reinterpret_cast<const v4i*>(stage + r * 128 + (piece ^ ((r >> 1) & 7)) * 16);
        }
    }
}

template <typename S, int MODE, bool BF16>
__global__ __launch_bounds__(64 * S::NW) void gemm_block_kernel(BlockGemmArgs a) {
    __shared__ __align__(1024) int8_t ring[2 * S::kStageBytes];
    __shared__ float s_sa[2 * S::kSa];
    __shared__ float s_sb[2 * kMaxKb];
    constexpr int chans = MODE == kGateUp ? S::BN / 2 : S::BN;  // output channels of a tile
    const int tiles_n = (a.N + chans - 1) / chans;
    Tile t;
    if constexpr (MODE == kDense) {
        constexpr int kGroupM = 4;  // tile rows that share a weight panel in L2
        const int tiles_m = (int)(((int64_t)a.M + a.tile_rows - 1) / a.tile_rows);
        const int L = xcd_order(blockIdx.x, tiles_m * tiles_n);
        const int first = L / (kGroupM * tiles_n) * kGroupM;
        const int gsz = min(tiles_m - first, kGroupM), in = L - first * tiles_n;
        t.row0 = (first + in % gsz) * a.tile_rows;
        t.n0 = in / gsz * chans;
        t.rows = min(a.tile_rows, a.M - t.row0);
        t.e = 0;
    } else {
        const int total = a.tiles[0] * tiles_n;
        if ((int)blockIdx.x >= total) return;
        const int L = xcd_order(blockIdx.x, total);
        const int32_t* at = a.tiles + 4 + 4 * (L / tiles_n);
        t.e = __builtin_amdgcn_readfirstlane(at[0]);
        t.row0 = __builtin_amdgcn_readfirstlane(at[1]);
        t.rows = __builtin_amdgcn_readfirstlane(at[2]);
        t.n0 = L % tiles_n * chans;
    }
    // as few row tiles per wave as the rows need
    constexpr int kRows = 16 * S::WM;
    if constexpr (S::kMaxMT == 8) {
        if (t.rows > 6 * kRows)
            tile_body<S, MODE, BF16, 8>(a, t, ring, s_sa, s_sb);
        else if (t.rows > 4 * kRows)
            tile_body<S, MODE, BF16, 6>(a, t, ring, s_sa, s_sb);
        else if (t.rows > 2 * kRows)
            tile_body<S, MODE, BF16, 4>(a, t, ring, s_sa, s_sb);
        else
            tile_body<S, MODE, BF16, 2>(a, t, ring, s_sa, s_sb);
    } else {
        tile_body<S, MODE, BF16, S::kMaxMT>(a, t, ring, s_sa, s_sb);
    }
}

typedef Shape<2, 4, 8> TileBig;    // up to 256 rows, 8 waves
typedef Shape<1, 4, 2> TileSmall;  // up to 32 rows, 4 waves

template <typename S, int MODE>
hipError_t launch(const BlockGemmArgs& a, int64_t tiles_m, hipStream_t stream) {
    const int chans = MODE == kGateUp ? S::BN / 2 : S::BN;
    const int64_t grid = tiles_m * ((a.N + chans - 1) / chans);
    if (grid > kMaxGrid) return hipErrorInvalidValue;
    if (a.bf16 && MODE == kDense)
        gemm_block_kernel<S, MODE, true><<<dim3((unsigned)grid), 64 * S::NW, 0, stream>>>(a);
    else
        gemm_block_kernel<S, MODE, false><<<dim3((unsigned)grid), 64 * S::NW, 0, stream>>>(a);
    return hipGetLastError();
}

// Rows of a dense product's tiles: 64, 128, 192 or 256, whichever takes the least
// time in rounds of the 256 CUs.  A tile's K stage is bound by LDS traffic: the
// weights' 96 KiB (written once, read by both wave rows) and 40 KiB for each 64
// rows.
int dense_tile_rows(int64_t M, int64_t N) {
    const int64_t tiles_n = (N + TileBig::BN - 1) / TileBig::BN;
    int best = 256;
    int64_t least = INT64_MAX;
    for (int rows = 256; rows >= 64; rows -= 64) {
        const int64_t rounds = ((M + rows - 1) / rows * tiles_n + 255) / 256;
        const int64_t time = rounds * (96 + 40 * (rows / 64));
        if (time < least) {
            least = time;
            best = rows;
        }
    }
    return best;
}

}  // namespace

size_t gemm_block_workspace(int64_t, int64_t, int64_t) { return 0; }

hipError_t launch_gemm_block(const BlockGemmArgs& in, void* workspace, hipStream_t stream) {
    (void)workspace;
    if (gemm_block_streams(in.M, in.N, in.K)) return launch_gemm_block_stream(in, stream);
    BlockGemmArgs a = in;
    a.tile_rows = dense_tile_rows(in.M, in.N);
    // row blocks of the activations small enough for one launch's grid
    const int64_t tiles_n = ((int64_t)a.N + TileBig::BN - 1) / TileBig::BN;
    const int64_t most = kMaxGrid / tiles_n * a.tile_rows;
    for (int64_t m = 0; m < in.M; m += most) {
        a.M = (int)(in.M - m < most ? in.M - m : most);
        a.CA = in.CA + m * a.K;
        a.SCA = in.SCA + m;
        a.Y = in.Y + m * a.N;
        const hipError_t e = launch<TileBig, kDense>(a, ((int64_t)a.M + a.tile_rows - 1) / a.tile_rows, stream);
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

int grouped_tile_rows(int64_t pairs, int E) { return pairs / E > 48 ? TileBig::BM : TileSmall::BM; }

hipError_t launch_experts_gate_up(const BlockGemmArgs& a, int tile_rows, int64_t max_tiles, hipStream_t stream) {
    if (tile_rows == TileBig::BM) return launch<TileBig, kGateUp>(a, max_tiles, stream);
    return launch<TileSmall, kGateUp>(a, max_tiles, stream);
}

hipError_t launch_experts_down(const BlockGemmArgs& a, int tile_rows, int64_t max_tiles, hipStream_t stream) {
    if (tile_rows == TileBig::BM) return launch<TileBig, kDown>(a, max_tiles, stream);
    return launch<TileSmall, kDown>(a, max_tiles, stream);
}

}  // namespace llmint8

// MXFP4: BF16 <-> 4-bit E2M1 codes with one power-of-two E8M0 scale per 32 elements, rowwise and/or
// columnwise, scales raw or in the tensor-core layout.
//
// The same microscaling rule, blocks, scale bytes and scale layout as the library's MXFP8 (OCP MX v1.0,
// whose MXFP4 has emax 2): per 32-block e = floor(log2 amax) - 2 clamped to [-127, 127], scale byte
// e + 127, an all-zero block byte 0; code = round-to-nearest-even(x * 2^-e) on the magnitudes 0, 0.5, 1,
// 1.5, 2, 3, 4, 6, saturated at 6, signed zero kept; two codes per byte, the even element in the low four
// bits. E2M1 has no NaN: a block holding NaN or an infinity gets scale byte 0xFF, which makes every value
// NaN, and codes sign | 7. x * 2^-e is exact in fp32 and one cvt.rn.satfinite rounds it.
//
// Both directions are bound by HBM: 2 bytes read and 17/32 bytes written per element and direction.
//
// This file must not be compiled with flush-to-zero: BF16 subnormals scaled by 2^127 are normal codes.
#pragma once
#include <cstdint>

#include "fastdiv.cuh"
#include "quantize.cuh"

namespace mx {

// Largest magnitude bits (0 .. 0x7FFF) of a block of 32.
__device__ __forceinline__ uint32_t block_absmax(const Block32& b) {
    uint32_t m = bf16x2_absmax(bf16x2_absmax(b.v[0].x, b.v[0].y), bf16x2_absmax(b.v[0].z, b.v[0].w));
#pragma unroll
    for (int j = 1; j < 4; ++j)
        m = bf16x2_absmax(m, bf16x2_absmax(bf16x2_absmax(b.v[j].x, b.v[j].y), bf16x2_absmax(b.v[j].z, b.v[j].w)));
    m &= 0x7FFF7FFFu;
    return max(m & 0xFFFFu, m >> 16);
}

// Scale byte from the largest BF16 magnitude bits: biased exponent - 2, at least 0.
__device__ __forceinline__ uint32_t fp4_scale_byte(uint32_t amax_bits) {
    if (amax_bits >= 0x7F80u) return 0xFFu;
    const int E = static_cast<int>(amax_bits >> 7);
    return static_cast<uint32_t>(E > 2 ? E - 2 : 0);
}

// Eight fp32 bit patterns (e[0] in the lowest four bits of the result) scaled by the packed pair inv2.
__device__ __forceinline__ uint32_t fp4_enc_oct(const uint32_t (&e)[8], uint64_t inv2) {
    uint32_t r;
    asm("{\n\t.reg .b64 x0, x1, x2, x3;\n\t.reg .f32 l0, h0, l1, h1, l2, h2, l3, h3;\n\t.reg .b8 c0, c1, c2, c3;\n\t"
        "mov.b64 x0, {%1, %2};\n\tmov.b64 x1, {%3, %4};\n\tmov.b64 x2, {%5, %6};\n\tmov.b64 x3, {%7, %8};\n\t"
        "mul.rn.f32x2 x0, x0, %9;\n\tmul.rn.f32x2 x1, x1, %9;\n\tmul.rn.f32x2 x2, x2, %9;\n\tmul.rn.f32x2 x3, x3, %9;\n\t"
        "mov.b64 {l0, h0}, x0;\n\tmov.b64 {l1, h1}, x1;\n\tmov.b64 {l2, h2}, x2;\n\tmov.b64 {l3, h3}, x3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c0, h0, l0;\n\tcvt.rn.satfinite.e2m1x2.f32 c1, h1, l1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c2, h2, l2;\n\tcvt.rn.satfinite.e2m1x2.f32 c3, h3, l3;\n\t"
        "mov.b32 %0, {c0, c1, c2, c3};\n\t}"
        : "=r"(r)
        : "r"(e[0]), "r"(e[1]), "r"(e[2]), "r"(e[3]), "r"(e[4]), "r"(e[5]), "r"(e[6]), "r"(e[7]), "l"(inv2));
    return r;
}

// Eight BF16 (one 16-byte chunk) -> eight codes in one word.
__device__ __forceinline__ uint32_t fp4_encode_chunk(const uint4 v, uint64_t inv2) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t e[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        e[2 * i] = w[i] << 16;
        e[2 * i + 1] = w[i] & 0xFFFF0000u;
    }
    return fp4_enc_oct(e, inv2);
}
// NaN or Inf in the block: every code is sign | 7.
__device__ __forceinline__ uint32_t fp4_special_chunk(const uint4 v) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t r = 0x77777777u;
#pragma unroll
    for (int i = 0; i < 4; ++i) r |= ((w[i] >> 12) & 8u) << (8 * i) | (w[i] >> 31) << (8 * i + 7);
    return r;
}

// The scale byte's special value is looked at once per block, behind the encoding (with a test per chunk the rowwise
// quantizer took 22.2 us for 12288 x 4096, like this 21.7).
__device__ __forceinline__ uint4 fp4_encode_block(const Block32& b, uint32_t s) {
    const uint64_t inv2 = inv_scale2(s);
    uint4 o = make_uint4(fp4_encode_chunk(b.v[0], inv2), fp4_encode_chunk(b.v[1], inv2),
                         fp4_encode_chunk(b.v[2], inv2), fp4_encode_chunk(b.v[3], inv2));
    if (s == 0xFFu)
        o = make_uint4(fp4_special_chunk(b.v[0]), fp4_special_chunk(b.v[1]), fp4_special_chunk(b.v[2]),
                       fp4_special_chunk(b.v[3]));
    return o;
}

// The 32 BF16 of one column (the low or the high halves of w[0..31]) -> 16 bytes, row i in nibble i.
__device__ __forceinline__ uint4 fp4_encode_col32(const uint32_t (&w)[32], uint32_t s, bool hi) {
    uint32_t o[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        uint32_t e[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) e[i] = hi ? (w[8 * q + i] & 0xFFFF0000u) : (w[8 * q + i] << 16);
        if (s != 0xFFu) {
            o[q] = fp4_enc_oct(e, inv_scale2(s));
        } else {
            o[q] = 0x77777777u;
#pragma unroll
            for (int i = 0; i < 8; ++i) o[q] |= (e[i] >> 31) << (4 * i + 3);
        }
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
}

// Raw or swizzled scale block of one 128 x 128 tile, from its 512-byte image in shared memory.
// rows x blocks: the scale matrix; rt, bt: the tile's row tile and block tile; lane16: 0 .. 127.
__device__ __forceinline__ void fp4_store_scales(uint8_t* s, const uint8_t* atom, bool swz, int64_t rows, int64_t blocks,
                                                 int64_t rt, int64_t bt, int64_t btiles, int lane128) {
    if (swz) {
        if (lane128 < 32)
            reinterpret_cast<uint4*>(s + (rt * btiles + bt) * 512)[lane128] = reinterpret_cast<const uint4*>(atom)[lane128];
    } else {
        const int64_t r = rt * 128 + lane128;
        const int nb = static_cast<int>(blocks - bt * 4 < 4 ? blocks - bt * 4 : 4);
        if (r < rows)
            for (int q = 0; q < nb; ++q)
                s[r * blocks + bt * 4 + q] = atom[(lane128 & 31) * 16 + (lane128 >> 5) * 4 + q];
    }
}

struct Fp4Args {
    QTensor t;                // x, q_row / q_col (packed codes), s_row / s_col, sizes, tile counts
    int swz;
    int64_t total_tiles;
};

// A CTA walks a contiguous range of 128 x 128 tiles. Thread t owns the 32-blocks (row t / 4, K-block
// t mod 4) and (row 64 + t / 4, same) of a tile, so amax, scale and codes need no cross-lane exchange.
// The next tile's halves are loaded into the registers of the current halves as soon as those are encoded
// (and, for the columnwise direction, staged in shared memory), so loads stay in flight through the rest
// of the tile. For the columnwise copy thread t then owns columns 2 (t mod 64), +1 over one 32-row M-block.
// Three CTAs per SM (80 registers): 12288 x 4096 takes 21.7 us rowwise (127 MB, 5.8 TB/s), 26 us columnwise and
// 32.5 us for both (154 MB, 4.7 TB/s; two CTAs per SM: 22, 29 and 35 us), where issue slots are 60% busy.
template <bool ROW, bool COL>
__global__ void __launch_bounds__(kQThreads, 3) quantize_fp4_kernel(const __grid_constant__ Fp4Args a) {
    grid_wait();
    __shared__ __align__(128) uint8_t tile[COL ? kQTile * 256 : 16];
    __shared__ __align__(16) uint8_t atom_row[512];
    __shared__ __align__(16) uint8_t atom_col[512];
    const int tid = threadIdx.x;
    const uint32_t tile_s = smem_u32(tile);
    const QTensor& T = a.t;
    const int64_t t_begin = static_cast<int64_t>(blockIdx.x) * a.total_tiles / gridDim.x;
    const int64_t t_end = (static_cast<int64_t>(blockIdx.x) + 1) * a.total_tiles / gridDim.x;
    const int kb = tid & 3;
    Block32 cur[2];
    int mt = static_cast<int>(t_begin / T.tiles_k), kt = static_cast<int>(t_begin % T.tiles_k);
    auto fetch = [&](int m, int k, int h) {
        const int64_t row = static_cast<int64_t>(m) * kQTile + h * 64 + (tid >> 2);
        const int64_t col = static_cast<int64_t>(k) * kQTile + kb * 32;
        load_block<true>(T, row, col, row < T.M && col < T.K, cur[h]);
    };
    if (t_begin < t_end) {
        fetch(mt, kt, 0);
        fetch(mt, kt, 1);
    }
    for (int64_t t = t_begin; t < t_end; ++t) {
        const int64_t m0 = static_cast<int64_t>(mt) * kQTile, k0 = static_cast<int64_t>(kt) * kQTile;
        const bool last_k = kt + 1 == T.tiles_k;
        const int mn = last_k ? mt + 1 : mt, kn = last_k ? 0 : kt + 1;      // the next tile
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int r = h * 64 + (tid >> 2);
            const Block32& b = cur[h];
            if constexpr (COL) {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    st_shared_v4(tile_s + qtile_chunk(r, kb * 4 + j), b.v[j].x, b.v[j].y, b.v[j].z, b.v[j].w);
            }
            if constexpr (ROW) {
                const int64_t row = m0 + r, col = k0 + kb * 32;
                const bool valid = row < T.M && col < T.K;
                const uint32_t s = fp4_scale_byte(block_absmax(b));
                if (valid) *reinterpret_cast<uint4*>(T.q_row + (row * T.K + col) / 2) = fp4_encode_block(b, s);
                atom_row[(r & 31) * 16 + (r >> 5) * 4 + kb] = valid ? static_cast<uint8_t>(s) : 0;
            }
            if (t + 1 < t_end) fetch(mn, kn, h);
        }
        __syncthreads();
        if constexpr (COL) {
            const int cp = tid & 63, mb = tid >> 6;
            uint32_t w[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) w[i] = ld_shared_u32(tile_s + qtile_chunk(mb * 32 + i, cp >> 2) + (cp & 3) * 4);
            const uint32_t m = col_pair_absmax(w);
            const int64_t kc = k0 + 2 * cp, mr = m0 + 32 * mb;
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
                const uint32_t s = fp4_scale_byte(hh ? (m >> 16) : (m & 0xFFFFu));
                const bool ok = mr < T.M && kc + hh < T.K;       // M % 32 == 0: a block is all in or all out
                if (ok) *reinterpret_cast<uint4*>(T.q_col + ((kc + hh) * T.M + mr) / 2) = fp4_encode_col32(w, s, hh != 0);
                const int kk = 2 * cp + hh;
                atom_col[(kk & 31) * 16 + (kk >> 5) * 4 + mb] = ok ? static_cast<uint8_t>(s) : 0;
            }
            __syncthreads();
        }
        if constexpr (ROW)
            if (tid < 128) fp4_store_scales(T.s_row, atom_row, a.swz != 0, T.M, T.K / 32, mt, kt, T.tiles_k, tid);
        if constexpr (COL)
            if (tid >= 128) fp4_store_scales(T.s_col, atom_col, a.swz != 0, T.K, T.M / 32, kt, mt, T.tiles_m, tid - 128);
        __syncthreads();
        mt = mn;
        kt = kn;
    }
}

// Eight codes (element 0 in the lowest four bits) -> eight BF16 times the BF16 pair `scale2`. The magnitudes'
// high and low BF16 bytes come from two byte tables (prmt takes four nibbles as selectors), the signs from the
// codes' top bits. Exact: a code has two significant bits, and the smallest product, 0.5 * 2^-127, is a BF16
// subnormal, which the packed multiply keeps. Scale NaN gives NaN; a product past BF16's range (scale bytes
// above 252 only, which quantization never writes) gives an infinity.
__device__ __forceinline__ uint4 fp4_decode_word(uint32_t q, uint32_t scale2) {
    const uint32_t m = q & 0x77777777u;
    // Codes 0 .. 7:   0     .5    1     1.5   2     3     4     6
    //   BF16       0000  3F00  3F80  3FC0  4000  4040  4080  40C0
    const uint32_t hi0 = __byte_perm(0x3F3F3F00u, 0x40404040u, m), hi1 = __byte_perm(0x3F3F3F00u, 0x40404040u, m >> 16);
    const uint32_t lo0 = __byte_perm(0xC0800000u, 0xC0804000u, m), lo1 = __byte_perm(0xC0800000u, 0xC0804000u, m >> 16);
    uint32_t o[4] = {__byte_perm(lo0, hi0, 0x5140), __byte_perm(lo0, hi0, 0x7362), __byte_perm(lo1, hi1, 0x5140),
                     __byte_perm(lo1, hi1, 0x7362)};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t u = i == 0 ? q << 12 : (i == 1 ? q << 4 : (i == 2 ? q >> 4 : q >> 12));   // code 2 i at bits 12-15
        o[i] |= (u & 0x8000u) | ((u << 12) & 0x80000000u);
        asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(o[i]) : "r"(o[i]), "r"(scale2));
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
}

struct Fp4DeqArgs {
    const uint8_t* q;         // [M, K / 2]: this launch's rows start at row0
    const uint8_t* s;         // raw [M, K / 32] or the tensor-core layout
    uint16_t* out;            // BF16 [M, K], row stride ld
    int64_t row0, ld, kblocks, ctiles;
    uint32_t words;           // words of eight codes in this launch, < 2^31
    FastDiv words_per_row;
    int swz;
};

constexpr int kDeqWords = 4;          // words per thread

// One thread per word of eight codes (4 bytes in, 16 bytes out), 4 words apart by the block's width, so loads
// and stores of a warp are consecutive; the four threads of a block of 32 read the same scale byte. Bound by
// HBM: 196 608 x 4096 takes 334 us, 6.1 TB/s of which 4.8 are written (a fill of 2 GB reaches 3.9); 12288 x 4096 24 us,
// 5.3 TB/s, where the launch and the last stores weigh.
__global__ void __launch_bounds__(256) dequantize_fp4_kernel(const __grid_constant__ Fp4DeqArgs a) {
    grid_wait();
    const uint32_t i0 = blockIdx.x * (256u * kDeqWords) + threadIdx.x;
    const uint8_t* qs = a.q + a.row0 * a.kblocks * 16;
    uint32_t q[kDeqWords], s[kDeqWords];
    int64_t at[kDeqWords];
#pragma unroll
    for (int j = 0; j < kDeqWords; ++j) {
        const uint32_t i = i0 + 256u * j;
        if (i < a.words) {
            const uint32_t rl = a.words_per_row.div(i), w = i - rl * a.words_per_row.d;     // row, word in it
            const int64_t r = a.row0 + rl, c = w >> 2;
            q[j] = reinterpret_cast<const uint32_t*>(qs)[i];
            s[j] = a.s[a.swz ? ((r >> 7) * a.ctiles + (c >> 2)) * 512 + (r & 31) * 16 + ((r & 127) >> 5) * 4 + (c & 3)
                             : r * a.kblocks + c];
            at[j] = r * a.ld + static_cast<int64_t>(w) * 8;
        }
    }
#pragma unroll
    for (int j = 0; j < kDeqWords; ++j)
        if (i0 + 256u * j < a.words) {
            const uint32_t f = s[j] == 0xFFu ? 0x7FC0u : (s[j] ? s[j] << 7 : 0x0040u);      // 2^(s - 127)
            *reinterpret_cast<uint4*>(a.out + at[j]) = fp4_decode_word(q[j], f | (f << 16));
        }
}

}  // namespace mx

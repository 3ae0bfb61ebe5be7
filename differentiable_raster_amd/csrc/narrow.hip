// The backward of a narrow linear map or gated unit (x of at most 64 or 128 columns, at most 256 weight rows)
// over many rows in one pass: per block of 64 rows the pre-activation is computed again, dz takes its place in
// LDS, and dx and the block's share of dweight come from there.
//
//   z = x W^T + b,  dz = dy act'(z)  (gated: dgate = dh u act'(g), dup = dh act(g)),
//   dx = dz W,  dW = sum over rows of dz^T x,  db = sum over rows of dz.
//
// Such a map is bound by memory: the tiled products would write dz (four times the bytes of x for 64 columns
// and 256 weight rows) and read it and x twice more.  Here x and dy are read once, dx is written once, the
// weights stay in registers as fragments of both products, and dW stays in the accumulators of a persistent
// workgroup, whose share is added up afterwards in a fixed order.
#include <type_traits>

#include "elem.h"
#include "neural.h"

namespace gsmi {
namespace {

constexpr int kRows = 64, kThreads = 512;

struct Bf16 {
    static constexpr int type = GS_TYPE_BF16;
    static __device__ __forceinline__ f32x4 mma(u32x4 a, u32x4 b, f32x4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
    }
};
struct F16 {
    static constexpr int type = GS_TYPE_F16;
    static __device__ __forceinline__ f32x4 mma(u32x4 a, u32x4 b, f32x4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
    }
};

// An array of rows of RB bytes in LDS, read along its rows and, transposed, along its columns: the 32-byte
// granule g of row r is kept at g ^ swizzle(r), so that neither way makes the rows of one read meet in a bank.
template <int RB>
struct Rows {
    static __device__ __forceinline__ int swizzle(int r) { return RB == 128 ? (r >> 1) & 3 : r & 7; }
    static __device__ __forceinline__ int at(int r, int byte) { return r * RB + (((byte >> 5) ^ swizzle(r)) << 5) + (byte & 31); }
    // 16 rows from r0 on, 32 columns from 32 kk on: lane l holds row l & 15, 8 columns of its quarter
    static __device__ __forceinline__ u32x4 along(const char* p, int r0, int kk, int lane) {
        return *reinterpret_cast<const u32x4*>(p + at(r0 + (lane & 15), kk * 64 + (lane >> 4) * 16));
    }
    // 16 columns (granule g), summed over 32 rows from 32 kk on: lane l holds column l & 15, 8 rows of its quarter
    static __device__ __forceinline__ u32x4 across(const char* p, int g, int kk, int lane) {
        const int l = lane & 15, r = kk * 32 + (lane >> 4) * 8 + (l >> 2), b = g * 32 + (l & 3) * 8;
        typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
        const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(p + at(r, b)));
        const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(p + at(r + 4, b)));
        const u32x2 u = __builtin_bit_cast(u32x2, lo), v = __builtin_bit_cast(u32x2, hi);
        return u32x4{u[0], u[1], v[0], v[1]};
    }
};

enum NarrowKind { kPlain = 0, kActivated = 1, kPaired = 2 };

// Workgroups that share a CU: two where the fragments, accumulators and dy fit 128 registers.
constexpr int per_cu(int kp, int np, int kind) { return kp * np == 64 * 64 || (kp * np == 64 * 128 && kind == kPlain) ? 2 : 1; }

// KP columns of x and NP weight rows at most; the paired kind keeps gates in rows 0..NP/2-1 and ups above.
template <class T, int KP, int NP, int KIND>
__global__ __launch_bounds__(kThreads, 2 * per_cu(KP, NP, KIND)) void narrow_kernel(NarrowArgs a) {
#ifdef __HIP_DEVICE_COMPILE__
    constexpr bool PAIRED = KIND == kPaired;
    typedef Rows<KP * 2> X;
    typedef Rows<NP * 2> Z;
    constexpr int W_BYTES = NP * KP * 2, Z_BYTES = kRows * NP * 2;
    __shared__ __align__(1024) char x0[kRows * KP * 2], x1[kRows * KP * 2];
    __shared__ __align__(1024) char zs[W_BYTES > Z_BYTES ? W_BYTES : Z_BYTES];  // the weights at first
    typedef __attribute__((address_space(3))) void lds_void;

    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), q = lane >> 4, l = lane & 15;
    const int32_t nblk = (int32_t)(((int64_t)a.rows + kRows - 1) / kRows);
    const int32_t H = PAIRED ? a.n / 2 : a.n;
    // weight row of LDS row n, or -1
    auto source = [&](int n) {
        if (!PAIRED) return n < H ? n : -1;
        const int half = n / (NP / 2), k = n % (NP / 2);
        return k < H ? half * H + k : -1;
    };

    // ---- roles of the waves ----
    constexpr int PF = PAIRED ? NP / 32 : NP / 16;           // columns of z in blocks of 16 (pairs)
    constexpr int CZ = PF > 8 ? PF / 8 : 1, WPF = PF < 8 ? 8 / PF : 1, RZ = 4 / WPF;
    constexpr int KF = KP / 16, WPK = 8 / KF, RX = 4 / WPK;  // columns of dx; waves per column; row blocks per wave
    constexpr int NF = NP / 16, NW = NF >= 8 ? NF / 8 : 1, KW = NF >= 8 ? KF : KF * NF / 8;  // dW blocks of a wave
    const int cz0 = PF >= 8 ? wave * CZ : wave % PF, rz0 = PF >= 8 ? 0 : wave / PF * RZ;
    const int kx = wave % KF, rx0 = wave / KF * RX;
    const int nw0 = NF >= 8 ? wave * NW : wave % NF, kw0 = NF >= 8 ? 0 : wave / NF * KW;

    // ---- the weights, once: through LDS into the fragments that this wave needs of them ----
    for (int id = tid; id < NP * (KP / 8); id += kThreads) {
        const int n = id / (KP / 8), c = id % (KP / 8), s = source(n);
        u32x4 v = {0u, 0u, 0u, 0u};
        if (s >= 0 && c * 8 < a.k) v = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(a.w) + (int64_t)s * a.ldw + c * 8);
        *reinterpret_cast<u32x4*>(zs + X::at(n, c * 16)) = v;
    }
    __syncthreads();
    u32x4 wz[CZ][PAIRED ? 2 : 1][KP / 32], wx[NP / 32];
    float bias[CZ][PAIRED ? 2 : 1][4];
#pragma unroll
    for (int c = 0; c < CZ; c++)
#pragma unroll
        for (int h = 0; h < (PAIRED ? 2 : 1); h++) {
            const int n0 = h * (NP / 2) + (cz0 + c) * 16;
#pragma unroll
            for (int kk = 0; kk < KP / 32; kk++) wz[c][h][kk] = X::along(zs, n0, kk, lane);
#pragma unroll
            for (int k = 0; k < 4; k++) {
                const int s = source(n0 + q * 4 + k);
                bias[c][h][k] = a.bias && s >= 0 ? a.bias[s] : 0.0f;
            }
        }
#pragma unroll
    for (int kk = 0; kk < NP / 32; kk++) wx[kk] = X::across(zs, kx, kk, lane);

    f32x4 dw[NW][KW];
    float db[CZ][PAIRED ? 2 : 1][4];
#pragma unroll
    for (int n = 0; n < NW; n++)
#pragma unroll
        for (int k = 0; k < KW; k++) dw[n][k] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int c = 0; c < CZ; c++)
#pragma unroll
        for (int h = 0; h < (PAIRED ? 2 : 1); h++)
#pragma unroll
            for (int k = 0; k < 4; k++) db[c][h][k] = 0.0f;

    // ---- loads of a block: x to LDS without passing a register (rows past the end arrive as zeros), dy to registers
    constexpr int XN = kRows * KP * 2 / 16 / kThreads;
    auto fetch_x = [&](char* xs, int32_t blk) {
        const int64_t r0 = (int64_t)blk * kRows;
        const int32_t rows = a.rows - r0 < kRows ? (int32_t)(a.rows - r0) : kRows;
        const char* base = static_cast<const char*>(a.x) + r0 * a.ldx * 2;
        const __amdgpu_buffer_rsrc_t rs =
            __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(base), 0, (int32_t)(((int64_t)(rows - 1) * a.ldx + a.k) * 2), 0x00020000);
#pragma unroll
        for (int n = 0; n < XN; n++) {
            const int id = tid + n * kThreads, r = id / (KP / 8), slot = id % (KP / 8);
            const int c = ((slot >> 1) ^ X::swizzle(r)) * 2 + (slot & 1);
            const int32_t off = r < rows && c * 8 < a.k ? (int32_t)(r * a.ldx * 2 + c * 16) : 0x7FFFFFF0;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_void*)(xs + (n * kThreads + wave * 64) * 16), 16, off, 0, 0, 0);
        }
    };
    const bool vec = a.d_sj == 1 && (a.d_si & 3) == 0 && (H & 3) == 0;
    f32x4 dy[RZ][CZ];
    auto fetch_dy_as = [&](auto type, int32_t blk) {
#pragma unroll
        for (int r = 0; r < RZ; r++)
#pragma unroll
            for (int c = 0; c < CZ; c++) {
                const int64_t i = (int64_t)blk * kRows + (rz0 + r) * 16 + l;
                const int32_t j = (cz0 + c) * 16 + q * 4;
                const int64_t at = i * a.d_si + j * a.d_sj;
                f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
                if (i < a.rows && j < H) {
                    if (vec) {
                        v = load_elem4(a.dy, decltype(type)::value, at);
                    } else {
#pragma unroll
                        for (int k = 0; k < 4; k++)
                            if (j + k < H) v[k] = load_elem(a.dy, decltype(type)::value, at + k * a.d_sj);
                    }
                }
                dy[r][c] = v;
            }
    };
    auto fetch_dy = [&](int32_t blk) {
        if (a.dy_type == GS_TYPE_F32)
            fetch_dy_as(std::integral_constant<int, GS_TYPE_F32>(), blk);
        else if (a.dy_type == GS_TYPE_BF16)
            fetch_dy_as(std::integral_constant<int, GS_TYPE_BF16>(), blk);
        else
            fetch_dy_as(std::integral_constant<int, GS_TYPE_F16>(), blk);
    };

    auto block = [&](char* xs, char* next, int32_t blk) {
        __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0): this block's x is in LDS, which the barrier alone does not wait for
        __syncthreads();
        f32x4 d[RZ][CZ];
#pragma unroll
        for (int r = 0; r < RZ; r++)
#pragma unroll
            for (int c = 0; c < CZ; c++) d[r][c] = dy[r][c];
        int ln = lane;  // addresses are computed again per block: held over the loop they cost more than they save
        asm volatile("" : "+v"(ln));
        const int32_t after = blk + gridDim.x;
        if (after < nblk) {
            fetch_x(next, after);
            fetch_dy(after);
        }
        // dz into LDS
        f32x4 z[RZ][CZ], u[RZ][CZ];
        if (KIND != kPlain) {
#pragma unroll
            for (int r = 0; r < RZ; r++) {
#pragma unroll
                for (int c = 0; c < CZ; c++)
#pragma unroll
                    for (int k = 0; k < 4; k++) {
                        z[r][c][k] = bias[c][0][k];
                        u[r][c][k] = bias[c][PAIRED ? 1 : 0][k];
                    }
#pragma unroll
                for (int kk = 0; kk < KP / 32; kk++) {
                    const u32x4 fx = X::along(xs, (rz0 + r) * 16, kk, ln);
#pragma unroll
                    for (int c = 0; c < CZ; c++) {
                        z[r][c] = T::mma(wz[c][0][kk], fx, z[r][c]);
                        if (PAIRED) u[r][c] = T::mma(wz[c][PAIRED ? 1 : 0][kk], fx, u[r][c]);
                    }
                }
            }
        }
        auto finish = [&](auto act) {
#pragma unroll
            for (int r = 0; r < RZ; r++) {
                const int row = (rz0 + r) * 16 + (ln & 15);
                const bool in = (int64_t)blk * kRows + row < a.rows;
#pragma unroll
                for (int c = 0; c < CZ; c++) {
                    const int j = (cz0 + c) * 16 + (ln >> 4) * 4;
                    float dg[4], du[4];
#pragma unroll
                    for (int k = 0; k < 4; k++) {
                        float v = 0.0f, dv = 1.0f;
                        if (KIND != kPlain) act_both(z[r][c][k], decltype(act)::value, v, dv);
                        const bool keep = in && j + k < H;
                        dg[k] = PAIRED ? d[r][c][k] * u[r][c][k] * dv : d[r][c][k] * dv;
                        dg[k] = keep ? dg[k] : 0.0f;
                        db[c][0][k] += dg[k];
                        if (PAIRED) {
                            du[k] = keep ? d[r][c][k] * v : 0.0f;
                            db[c][PAIRED ? 1 : 0][k] += du[k];
                        }
                    }
                    *reinterpret_cast<u32x2*>(zs + Z::at(row, j * 2)) = u32x2{pack2(dg[0], dg[1], T::type), pack2(dg[2], dg[3], T::type)};
                    if (PAIRED)
                        *reinterpret_cast<u32x2*>(zs + Z::at(row, NP + j * 2)) =
                            u32x2{pack2(du[0], du[1], T::type), pack2(du[2], du[3], T::type)};
                }
            }
        };
        if (KIND == kPlain || a.act == GS_ACT_NONE)
            finish(std::integral_constant<int, GS_ACT_NONE>());
        else if (a.act == GS_ACT_SILU)
            finish(std::integral_constant<int, GS_ACT_SILU>());
        else if (a.act == GS_ACT_GELU)
            finish(std::integral_constant<int, GS_ACT_GELU>());
        else
            finish(std::integral_constant<int, GS_ACT_RELU>());
        __syncthreads();
        // dx: this wave's 16 columns of some of the rows
        if (a.dx) {
#pragma unroll
            for (int r = 0; r < RX; r++) {
                f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int kk = 0; kk < NP / 32; kk++) acc = T::mma(wx[kk], Z::along(zs, (rx0 + r) * 16, kk, ln), acc);
                const int64_t i = (int64_t)blk * kRows + (rx0 + r) * 16 + (ln & 15);
                const int32_t j = kx * 16 + (ln >> 4) * 4;
                if (i < a.rows && j < a.k) {
                    uint16_t* o = static_cast<uint16_t*>(a.dx) + i * a.ld_dx + j;
                    if (a.dx_vec) {
                        *reinterpret_cast<u32x2*>(o) = u32x2{pack2(acc[0], acc[1], T::type), pack2(acc[2], acc[3], T::type)};
                    } else {
                        for (int k = 0; k < 4; k++) o[k] = (uint16_t)pack2(acc[k], 0.0f, T::type);  // k is a multiple of 8
                    }
                }
            }
        }
        if (a.dw_partial) {
#pragma unroll
            for (int kk = 0; kk < kRows / 32; kk++) {
                u32x4 fn[NW], fk[KW];
#pragma unroll
                for (int n = 0; n < NW; n++) fn[n] = Z::across(zs, nw0 + n, kk, ln);
#pragma unroll
                for (int k = 0; k < KW; k++) fk[k] = X::across(xs, kw0 + k, kk, ln);
#pragma unroll
                for (int n = 0; n < NW; n++)
#pragma unroll
                    for (int k = 0; k < KW; k++) dw[n][k] = T::mma(fk[k], fn[n], dw[n][k]);
            }
        }
    };
    int32_t blk = blockIdx.x;
    __syncthreads();  // the weights' fragments are read: their memory is dz's from here on
    if (blk < nblk) {
        fetch_x(x0, blk);
        fetch_dy(blk);
    }
    for (; blk < nblk; blk += 2 * gridDim.x) {
        block(x0, x1, blk);
        if (blk + (int32_t)gridDim.x < nblk) block(x1, x0, blk + gridDim.x);
    }

    // ---- this workgroup's shares ----
    if (a.dw_partial) {
        float* o = a.dw_partial + (int64_t)blockIdx.x * a.n * a.k;
#pragma unroll
        for (int n = 0; n < NW; n++) {
            const int s = source((nw0 + n) * 16 + l);
#pragma unroll
            for (int k = 0; k < KW; k++) {
                const int j = (kw0 + k) * 16 + q * 4;
                if (s >= 0 && j < a.k) *reinterpret_cast<f32x4*>(o + (int64_t)s * a.k + j) = dw[n][k];
            }
        }
    }
    if (a.db_partial) {
        float* o = a.db_partial + ((int64_t)blockIdx.x * WPF + (PF >= 8 ? 0 : wave / PF)) * a.n;
#pragma unroll
        for (int c = 0; c < CZ; c++)
#pragma unroll
            for (int h = 0; h < (PAIRED ? 2 : 1); h++)
#pragma unroll
                for (int k = 0; k < 4; k++) {
                    float s = db[c][h][k];
#pragma unroll
                    for (int m = 1; m < 16; m <<= 1) s += __shfl_xor(s, m);
                    const int n = source(h * (NP / 2) + (cz0 + c) * 16 + q * 4 + k);
                    if (l == 0 && n >= 0) o[n] = s;
                }
    }
#endif
}

template <class T, int KP, int NP>
hipError_t launch_size(const NarrowArgs& a, bool gated, int groups, hipStream_t s) {
    if (gated)
        hipLaunchKernelGGL((narrow_kernel<T, KP, NP, kPaired>), dim3(groups), dim3(kThreads), 0, s, a);
    else if (a.act != GS_ACT_NONE)
        hipLaunchKernelGGL((narrow_kernel<T, KP, NP, kActivated>), dim3(groups), dim3(kThreads), 0, s, a);
    else
        hipLaunchKernelGGL((narrow_kernel<T, KP, NP, kPlain>), dim3(groups), dim3(kThreads), 0, s, a);
    return hipGetLastError();
}

template <class T>
hipError_t launch_type(const NarrowArgs& a, bool gated, const NarrowShape& p, hipStream_t s) {
    if (p.kp == 64) {
        if (p.np == 64) return launch_size<T, 64, 64>(a, gated, p.groups, s);
        if (p.np == 128) return launch_size<T, 64, 128>(a, gated, p.groups, s);
        return launch_size<T, 64, 256>(a, gated, p.groups, s);
    }
    if (p.np == 64) return launch_size<T, 128, 64>(a, gated, p.groups, s);
    return launch_size<T, 128, 128>(a, gated, p.groups, s);
}

}  // namespace

NarrowShape narrow_shape(int64_t rows, int64_t k, int64_t n, bool gated, bool activated) {
    NarrowShape p{0, 0, 0, 0};
    if (rows < 4096 || k > 128) return p;
    const int64_t width = gated ? 2 * ((n / 2 + 15) / 16 * 16) : n;
    if (width > (k <= 64 ? 256 : 128)) return p;
    p.kp = k <= 64 ? 64 : 128;
    p.np = width <= 64 ? 64 : width <= 128 ? 128 : 256;
    const int64_t blocks = (rows + kRows - 1) / kRows;
    const int most = 256 * per_cu(p.kp, p.np, gated ? kPaired : activated ? kActivated : kPlain);
    p.groups = (int)(blocks < most ? blocks : most);
    const int pf = gated ? p.np / 32 : p.np / 16;
    p.db_rows = p.groups * (pf < 8 ? 8 / pf : 1);
    return p;
}

hipError_t launch_narrow(int type, const NarrowArgs& a, bool gated, const NarrowShape& p, hipStream_t s) {
    return type == GS_TYPE_BF16 ? launch_type<Bf16>(a, gated, p, s) : launch_type<F16>(a, gated, p, s);
}

}  // namespace gsmi

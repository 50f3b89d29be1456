// selective_scan_bwd.cu -- the gradient of the selective state space scan (selective_scan.cu).
//
// With dy = d_out silu(z), and dh_t the gradient of the state after token t,
//   dh_t   = dy_t C_t + a_{t+1} dh_{t+1}          (from the last token back; + d_state_out there)
//   dC_t   = sum_d dy_t h_t                       (over the channels of a group)
//   dB_t   = sum_d dh_t dt_t u_t
//   dA     = sum_t dh_t a_t h_{t-1} dt_t
//   d dt_t = sum_n dh_t a_t h_{t-1} A + u_t sum_n dh_t B_t,   d delta_t = d dt_t sigmoid(delta_t + bias)
//   du_t   = D dy_t + dt_t sum_n dh_t B_t,   dz_t = d_out_t y_t silu'(z_t),   dD = sum dy_t u_t.
//
// The states h_t are needed from the last token back, so the forward keeps the state before every
// kScanChunk-th token; a block takes one sequence and a tile of channels (laid out over the lanes as
// in the forward), goes through the chunks from the last one, computes a chunk's 8 states and decay
// factors again in registers, and then steps back through them.  The sums over the channels of dB
// and dC are taken over a warp's channels by shuffles, over the block's warps in shared memory, and
// over the blocks of a group by a second kernel, in a fixed order; dA, dD and d bias are summed over
// the tokens in registers and over the sequences by that kernel too.
#include "seq_common.cuh"

namespace ttt {
namespace {

constexpr int kWarps = 8;
constexpr int kT = kScanChunk;

template <bool PAD>
__device__ __forceinline__ void load4(const float* p, int left, float (&h)[4]) {
    if constexpr (!PAD) {
        const float4 v = *reinterpret_cast<const float4*>(p);
        h[0] = v.x; h[1] = v.y; h[2] = v.z; h[3] = v.w;
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) h[i] = i < left ? p[i] : 0.f;
    }
}
template <bool PAD>
__device__ __forceinline__ void store4(float* p, int left, const float (&h)[4]) {
    if constexpr (!PAD) {
        *reinterpret_cast<float4*>(p) = make_float4(h[0], h[1], h[2], h[3]);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < left) p[i] = h[i];
    }
}

// The sums over a channel's P lanes of kT values (one a token): lane q ends with those of its tokens
// q, P + q, ... (P <= kT) or, with P = 2 kT lanes, of token q mod kT.
template <int P, int CPW>
__device__ __forceinline__ void token_sums(float (&v)[kT], int q, float (&out)[(kT + P - 1) / P]) {
    if constexpr (P <= kT) {
#pragma unroll
        for (int k = 0; k < kT / P; ++k) {
            float w[P];
#pragma unroll
            for (int j = 0; j < P; ++j) w[j] = v[k * P + j];
            out[k] = reduce_across<P, CPW>(w, q);
        }
    } else {
        const float s = reduce_across<kT, CPW>(v, q);
        out[0] = s + __shfl_xor_sync(0xffffffffu, s, kT * CPW);
    }
}

template <typename T, int P, bool PAD>
__global__ void __launch_bounds__(kWarps * 32) scan_bwd_kernel(const ScanBwdArgs a) {
    constexpr int CPW = 32 / P, CH = kWarps * CPW, NP = 4 * P;
    constexpr int K = (kT + P - 1) / P;              // tokens of a chunk that a lane finishes
    constexpr int BC = kT * 2 * NP;                  // values of B and C of a chunk
    constexpr int NB = (BC + kWarps * 32 - 1) / (kWarps * 32);
    constexpr int V = 64 / CPW;                      // of a lane's 2 kT 4 shares, those it sums over the channels
    __shared__ __align__(16) float sbc[BC];          // [token][B, C][n]
    __shared__ __align__(16) float4 sv[kWarps][kT][CPW];  // (dt, dt u, dy)
    __shared__ float red[kWarps][2][kT][NP];

    const int r = a.dim / a.groups;
    const int ct = blockIdx.x % (a.groups * a.tiles), g = ct / a.tiles, tile = ct % a.tiles;
    each_rest_row(a.s, blockIdx.x / (a.groups * a.tiles), a.s.n_seq, [&](long long row) {
        const int k = tile * CH + threadIdx.x;
        if (threadIdx.x < CH && k < r) {
            const long long at = row * a.dim + g * r + k;
            static_cast<T*>(a.du)[at] = static_cast<T*>(a.ddelta)[at] = from_f32<T>(0.f);
            if (a.dz) static_cast<T*>(a.dz)[at] = from_f32<T>(0.f);
        }
    });
    Piece p;
    find_piece(a.s, blockIdx.x / (a.groups * a.tiles), 1 << 30, p);  // the whole sequence

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, q = lane / CPW, c = lane % CPW;
    const int cg = tile * CH + warp * CPW + c;
    const bool live = cg < r;
    const int d = g * r + (live ? cg : r - 1);
    const int left = a.N - 4 * q;
    const bool mine = P <= kT || q < kT;             // this lane finishes tokens
    const long long hoff = static_cast<long long>(d) * a.N + 4 * q, hrow = static_cast<long long>(a.dim) * a.N;

    float A[4], A2[4], dA[4] = {0.f, 0.f, 0.f, 0.f}, dh[4] = {0.f, 0.f, 0.f, 0.f};
    load4<PAD>(a.A + hoff, left, A);
#pragma unroll
    for (int i = 0; i < 4; ++i) A2[i] = A[i] * kLog2e;
    if (a.d_state_out) load4<PAD>(a.d_state_out + p.b * hrow + hoff, left, dh);
    const float bias = a.bias ? a.bias[d] : 0.f, Dk = a.D ? a.D[d] : 0.f;
    float sum_D = 0.f, sum_bias = 0.f;

    const T* u = static_cast<const T*>(a.u) + p.row * a.su.b + p.t0 * a.su.t + d;
    const T* dl = static_cast<const T*>(a.delta) + p.row * a.sdt.b + p.t0 * a.sdt.t + d;
    const T* z = a.z ? static_cast<const T*>(a.z) + p.row * a.sz.b + p.t0 * a.sz.t + d : nullptr;
    const T* dout = static_cast<const T*>(a.d_out) + p.row * a.sdo.b + p.t0 * a.sdo.t + d;
    const T* Bm = static_cast<const T*>(a.B) + p.row * a.sB.b + p.t0 * a.sB.t + g * a.N;
    const T* Cm = static_cast<const T*>(a.C) + p.row * a.sC.b + p.t0 * a.sC.t + g * a.N;
    const long long row0 = p.row * a.s.L + p.t0;     // first row of the contiguous outputs
    T* du = static_cast<T*>(a.du) + row0 * a.dim + d;
    T* ddelta = static_cast<T*>(a.ddelta) + row0 * a.dim + d;
    T* dz = a.dz ? static_cast<T*>(a.dz) + row0 * a.dim + d : nullptr;
    const long long rows = a.s.cu ? a.s.L : a.s.n_seq * a.s.L;
    float* part_bc = a.part_bc + ((tile * rows + row0) * a.groups + g) * 2 * a.N;
    const long long chunk0 = a.s.cu ? slot_base(a.s.cu, p.b, a.s.L, kT) : p.b * ((a.s.L + kT - 1) / kT);
    const float* ckpt = a.ckpt + chunk0 * hrow + hoff;

    T ru[K], rd[K], rz[K], ro[K], rbc[NB];
    float h0[4];
    auto load_chunk = [&](int ch) {
        const int t0 = ch * kT;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int t = t0 + k * P + q;
            ru[k] = rd[k] = rz[k] = ro[k] = from_f32<T>(0.f);
            if (mine && t < p.len) {
                ru[k] = u[t * a.su.t];
                rd[k] = dl[t * a.sdt.t];
                ro[k] = dout[t * a.sdo.t];
                if (z) rz[k] = z[t * a.sz.t];
            }
        }
#pragma unroll
        for (int k = 0; k < NB; ++k) {
            const int e = k * kWarps * 32 + threadIdx.x, t = t0 + e / (2 * NP), n = e % NP;
            rbc[k] = from_f32<T>(0.f);
            if (e < BC && t < p.len && (!PAD || n < a.N))
                rbc[k] = (e / NP) & 1 ? Cm[t * a.sC.t + n] : Bm[t * a.sB.t + n];
        }
        load4<PAD>(ckpt + ch * hrow, left, h0);
    };

    const int chunks = (p.len + kT - 1) / kT;
    if (chunks > 0) load_chunk(chunks - 1);
    for (int ch = chunks - 1; ch >= 0; --ch) {
        const int t0 = ch * kT, n = min(kT, p.len - t0);
#pragma unroll
        for (int k = 0; k < NB; ++k) {
            const int e = k * kWarps * 32 + threadIdx.x;
            if (e < BC) sbc[e] = to_f32(rbc[k]);
        }
        float fu[K], fz[K], fo[K], fdy[K], fx[K], fdt[K], hs[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) hs[i] = h0[i];
#pragma unroll
        for (int k = 0; k < K; ++k) {
            fu[k] = to_f32(ru[k]);
            fz[k] = to_f32(rz[k]);
            fo[k] = to_f32(ro[k]);
            fx[k] = to_f32(rd[k]) + bias;
            fdt[k] = a.softplus ? softplus_f(fx[k]) : fx[k];
            if (k * P + q >= n) fdt[k] = 0.f;
            fdy[k] = z ? fo[k] * silu_f(fz[k]) : fo[k];
            if (mine) sv[warp][k * P + q][c] = make_float4(fdt[k], fdt[k] * fu[k], fdy[k], 0.f);
        }
        __syncthreads();  // B, C and the tokens' values; the last chunk's sums have been read
        if (ch > 0) load_chunk(ch - 1);

        // the chunk's decay factors and states
        float av[kT][4], hv[kT][4], y[kT], s1[kT], s2[kT];
#pragma unroll
        for (int t = 0; t < kT; ++t) {
            const float4 v = sv[warp][t][c];
            const float4 b4 = *reinterpret_cast<const float4*>(&sbc[(2 * t) * NP + 4 * q]);
            const float4 c4 = *reinterpret_cast<const float4*>(&sbc[(2 * t + 1) * NP + 4 * q]);
            const float b[4] = {b4.x, b4.y, b4.z, b4.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                av[t][i] = decay2(t < n ? v.x * A2[i] : 0.f);
                hv[t][i] = fmaf(av[t][i], t ? hv[t - 1][i] : hs[i], v.y * b[i]);
                if (PAD && i >= left) hv[t][i] = 0.f;
            }
            y[t] = fmaf(c4.x, hv[t][0], c4.y * hv[t][1]) + fmaf(c4.z, hv[t][2], c4.w * hv[t][3]);
        }
        // back through it
        float share[64];  // [dB, dC][token][n]
#pragma unroll
        for (int t = kT - 1; t >= 0; --t) {
            const float4 v = sv[warp][t][c];
            const float4 b4 = *reinterpret_cast<const float4*>(&sbc[(2 * t) * NP + 4 * q]);
            const float4 c4 = *reinterpret_cast<const float4*>(&sbc[(2 * t + 1) * NP + 4 * q]);
            const float b[4] = {b4.x, b4.y, b4.z, b4.w}, cc[4] = {c4.x, c4.y, c4.z, c4.w};
            s1[t] = s2[t] = 0.f;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float e = fmaf(v.z, cc[i], dh[i]);
                share[(kT + t) * 4 + i] = live ? v.z * hv[t][i] : 0.f;
                share[t * 4 + i] = live ? e * v.y : 0.f;
                dh[i] = e * av[t][i];
                const float m = dh[i] * (t ? hv[t - 1][i] : hs[i]);
                s1[t] = fmaf(e, b[i], s1[t]);
                s2[t] = fmaf(m, A[i], s2[t]);
                dA[i] = fmaf(m, v.x, dA[i]);
            }
        }
        float ys[K], s1s[K], s2s[K];
        token_sums<P, CPW>(s1, q, s1s);
        token_sums<P, CPW>(s2, q, s2s);
        if (z) token_sums<P, CPW>(y, q, ys);
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int t = k * P + q;
            if (mine && t < n) {
                const float gd = fmaf(fu[k], s1s[k], s2s[k]);
                const float gx = a.softplus ? gd * sigmoid_f(fx[k]) : gd;
                sum_bias += gx;
                sum_D = fmaf(fdy[k], fu[k], sum_D);
                if (live) {
                    const long long at = static_cast<long long>(t0 + t) * a.dim;
                    du[at] = from_f32<T>(fmaf(Dk, fdy[k], fdt[k] * s1s[k]));
                    ddelta[at] = from_f32<T>(gx);
                    if (z) dz[at] = from_f32<T>(fo[k] * fmaf(Dk, fu[k], ys[k]) * silu_grad_f(fz[k], sigmoid_f(fz[k])));
                }
            }
        }
        // the shares of dB and dC over the warp's channels: lane c ends with the shares V c .. V c + V - 1
#pragma unroll
        for (int w = CPW / 2, m = 32; w >= 1; w /= 2, m /= 2) {
#pragma unroll
            for (int i = 0; i < m; ++i) {
                const float send = (c & w) ? share[i] : share[i + m], keep = (c & w) ? share[i + m] : share[i];
                share[i] = keep + __shfl_xor_sync(0xffffffffu, send, w);
            }
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int e = c * V + i;
            (&red[warp][0][0][0])[(e / 4) * NP + 4 * q + e % 4] = share[i];
        }
        __syncthreads();
        // and over the block's warps
        for (int e = threadIdx.x; e < 2 * kT * NP; e += kWarps * 32) {
            const int which = e / (kT * NP), t = e / NP % kT, nn = e % NP;
            float s = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) s += red[w][which][t][nn];
            if (t < n && (!PAD || nn < a.N))
                part_bc[(static_cast<long long>(t0 + t) * a.groups * 2 + which) * a.N + nn] = s;
        }
    }
#pragma unroll
    for (int w = P / 2; w >= 1; w /= 2) {
        sum_D += __shfl_xor_sync(0xffffffffu, sum_D, w * CPW);
        sum_bias += __shfl_xor_sync(0xffffffffu, sum_bias, w * CPW);
    }
    if (live) {
        store4<PAD>(a.part_a + p.b * hrow + hoff, left, dA);
        if (a.d_state_in) store4<PAD>(a.d_state_in + p.b * hrow + hoff, left, dh);
        if (q == 0) {
            a.part_d[(2ll * p.b) * a.dim + d] = sum_D;
            a.part_d[(2ll * p.b + 1) * a.dim + d] = sum_bias;
        }
    }
}

// The sums over the channel tiles (dB, dC of every row) and over the sequences (dA, dD, d bias), in
// the order of the tiles and of the sequences.
template <typename T>
__global__ void __launch_bounds__(256) scan_bwd_sum_kernel(const ScanBwdArgs a, long long rows, long long n_bc,
                                                           long long n_a) {
    const long long i = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x;
    if (i < n_bc) {
        const long long per = rows * a.groups * 2 * a.N, row = i / (a.groups * 2 * a.N);
        bool in = true;
        if (a.s.cu) {
            in = row >= cu_at(a.s.cu, 0, a.s.L) && row < cu_at(a.s.cu, a.s.n_seq, a.s.L);
            if (!in && !a.s.zero_rest) return;
        }
        float s = 0.f;
        if (in)
            for (int k = 0; k < a.tiles; ++k) s += a.part_bc[k * per + i];
        const int n = static_cast<int>(i % a.N), which = static_cast<int>(i / a.N % 2);
        const long long g = i / (2 * a.N);
        (which ? static_cast<T*>(a.dC) : static_cast<T*>(a.dB))[g * a.N + n] = from_f32<T>(s);
    } else if (i < n_bc + n_a) {
        const long long e = i - n_bc;
        float s = 0.f;
        for (int b = 0; b < a.s.n_seq; ++b) s += a.part_a[b * n_a + e];
        a.dA[e] = s;
    } else if (i < n_bc + n_a + 2 * a.dim) {
        const int e = static_cast<int>(i - n_bc - n_a);
        float s = 0.f;
        for (int b = 0; b < a.s.n_seq; ++b) s += a.part_d[2ll * b * a.dim + e];
        float* out = e < a.dim ? a.dD : a.dbias;
        if (out) out[e % a.dim] = s;
    }
}

template <typename T, int P, bool PAD>
cudaError_t run(const ScanBwdArgs& a, cudaStream_t s) {
    const unsigned grid = static_cast<unsigned>(static_cast<long long>(a.s.n_seq) * a.groups * a.tiles);
    scan_bwd_kernel<T, P, PAD><<<grid, kWarps * 32, 0, s>>>(a);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    const long long rows = a.s.cu ? a.s.L : a.s.n_seq * a.s.L;
    const long long n_bc = rows * a.groups * 2 * a.N, n_a = static_cast<long long>(a.dim) * a.N;
    const long long n = n_bc + n_a + 2 * a.dim;
    scan_bwd_sum_kernel<T><<<static_cast<unsigned>((n + 255) / 256), 256, 0, s>>>(a, rows, n_bc, n_a);
    return cudaGetLastError();
}

template <typename T, int P>
cudaError_t pad(const ScanBwdArgs& a, cudaStream_t s) {
    return a.N == 4 * P ? run<T, P, false>(a, s) : run<T, P, true>(a, s);
}
template <typename T>
cudaError_t dispatch(const ScanBwdArgs& a, cudaStream_t s) {
    if (a.N <= 4) return pad<T, 1>(a, s);
    if (a.N <= 8) return pad<T, 2>(a, s);
    if (a.N <= 16) return pad<T, 4>(a, s);
    if (a.N <= 32) return pad<T, 8>(a, s);
    return pad<T, 16>(a, s);
}

}  // namespace

int scan_bwd_channels(int N) { return kWarps * 32 / (N <= 4 ? 1 : N <= 8 ? 2 : N <= 16 ? 4 : N <= 32 ? 8 : 16); }

cudaError_t launch_scan_bwd(const ScanBwdArgs& a, int dtype, cudaStream_t s) {
    return dtype == 0 ? dispatch<float>(a, s) : dispatch<__nv_bfloat16>(a, s);
}

}  // namespace ttt

// selective_scan.cu -- the selective state space scan over tokens, for prompts, and one token of it:
//
//   dt = softplus(delta + bias) (or delta + bias),   a = exp(dt A[d][n]),
//   h[d][n] = a h[d][n] + dt u[d] B[t][n],   y[d] = sum_n C[t][n] h[d][n] + D[d] u[d],
//   out[d] = y[d] silu(z[d])  (or y[d]),
//
// with B and C shared by the channels of a group.  The state stays in registers from a sequence's
// first token to its last: P lanes share a channel, each holding 4 of its N <= 4 P states, so a warp
// walks 32 / P channels down the tokens.
//
// What bounds it: a channel and token moves 4 elements (u, delta, z, out; 8 bytes in bf16) and takes
// N exponentials, on a unit that does 16 a cycle and SM, next to 4 N to 5 N multiplications.  At
// N = 16 the exponentials alone take about three times as long as the bytes.
//
// Each block takes one sequence and 8 * 32 / P channels of one group.  Tiles of 16 tokens: lane q of
// a channel's P lanes loads and finishes the tokens q, P + q, ... of the tile (their dt, dt u and the
// gate), and hands (dt, dt u) to the other lanes through shared memory; B and C of the tile lie in
// shared memory in float.  The sums over a channel's lanes are taken for P tokens at a time
// (reduce_across), which leaves each token's y with the lane that finishes it.
//
// Few sequences of many tokens leave most of the GPU idle, so those are cut into spans: a first
// launch runs every span but the last from a zero state (no outputs) and keeps its end state and its
// sum of dt; the second starts each span from the spans before it,
//   h = exp(A sum dt) h + end state of the span,
// and writes the outputs.  That is about 1.7 times the work, for as many times the blocks.
#include "seq_common.cuh"

namespace ttt {
namespace {

constexpr int kWarps = 8;
constexpr int kTile = 16;

enum Mode { kWhole, kSpanState, kSpanOut };

// Four states of a lane, n .. n + 3 of `N`; PAD: N is not 4 P, so the last lanes hold fewer.
template <bool PAD>
__device__ __forceinline__ void load_state(const float* p, int left, float (&h)[4]) {
    if constexpr (!PAD) {
        const float4 v = *reinterpret_cast<const float4*>(p);
        h[0] = v.x; h[1] = v.y; h[2] = v.z; h[3] = v.w;
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) h[i] = i < left ? p[i] : 0.f;
    }
}
template <bool PAD>
__device__ __forceinline__ void store_state(float* p, int left, const float (&h)[4]) {
    if constexpr (!PAD) {
        *reinterpret_cast<float4*>(p) = make_float4(h[0], h[1], h[2], h[3]);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < left) p[i] = h[i];
    }
}

template <typename T, int P, bool PAD, int MODE>
__global__ void __launch_bounds__(kWarps * 32) scan_kernel(const ScanArgs a) {
    constexpr int CPW = 32 / P, CH = kWarps * CPW, NP = 4 * P;
    constexpr int K = kTile / P;                     // tokens of a tile that a lane finishes
    constexpr int BC = kTile * 2 * NP;               // values of B and C of a tile
    constexpr int NB = (BC + kWarps * 32 - 1) / (kWarps * 32);
    __shared__ __align__(16) float sbc[2][BC];       // [token][B, C][n]
    __shared__ float2 sdt[kWarps][kTile][CPW];       // (dt, dt u)

    const int r = a.dim / a.groups, tiles = (r + CH - 1) / CH;
    const int ct = blockIdx.x % (a.groups * tiles), g = ct / tiles;
    Piece p;
    int first, last;
    if (!find_piece(a.s, blockIdx.x / (a.groups * tiles), a.span, p)) return;
    first = p.tile * a.span;
    last = min(first + a.span, p.len);
    if (MODE == kSpanState && p.tile > 0 && last == p.len) return;  // nothing starts from the last span

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, q = lane / CPW, c = lane % CPW;
    const int cg = (ct % tiles) * CH + warp * CPW + c;   // channel within the group
    const bool live = cg < r;
    const int d = g * r + (live ? cg : r - 1);
    const int left = a.N - 4 * q;
    const long long hoff = static_cast<long long>(d) * a.N + 4 * q, hrow = static_cast<long long>(a.dim) * a.N;

    float A2[4], h[4] = {0.f, 0.f, 0.f, 0.f};
    load_state<PAD>(a.A + hoff, left, A2);
#pragma unroll
    for (int i = 0; i < 4; ++i) A2[i] *= kLog2e;
    const float bias = a.bias ? a.bias[d] : 0.f, Dk = a.D ? a.D[d] : 0.f;

    const int page = page_of(a.pages, a.n_pages, p.b);
    if (MODE == kWhole || (MODE == kSpanState && p.tile == 0)) {
        if (a.state_in && page >= 0) load_state<PAD>(a.state_in + page * hrow + hoff, left, h);
        if (MODE == kSpanState && live) store_state<PAD>(a.seg_h0 + p.b * hrow + hoff, left, h);
        if (MODE == kSpanState && last == p.len) return;
    } else if (MODE == kSpanOut) {
        if (p.tile == 0) {
            load_state<PAD>(a.seg_h0 + p.b * hrow + hoff, left, h);
        } else {
            const int s0 = p.slot - p.tile;
            load_state<PAD>(a.seg_h + s0 * hrow + hoff, left, h);
            for (int s = s0 + 1; s < p.slot; ++s) {
                float e[4];
                load_state<PAD>(a.seg_h + s * hrow + hoff, left, e);
                const float sum = a.seg_dt[static_cast<long long>(s) * a.dim + d];
#pragma unroll
                for (int i = 0; i < 4; ++i) h[i] = fmaf(decay2(sum * A2[i]), h[i], e[i]);
            }
        }
    }

    const T* u = static_cast<const T*>(a.u) + p.row * a.su.b + p.t0 * a.su.t + d;
    const T* dl = static_cast<const T*>(a.delta) + p.row * a.sdt.b + p.t0 * a.sdt.t + d;
    const T* z = a.z ? static_cast<const T*>(a.z) + p.row * a.sz.b + p.t0 * a.sz.t + d : nullptr;
    const T* Bm = static_cast<const T*>(a.B) + p.row * a.sB.b + p.t0 * a.sB.t + g * a.N;
    const T* Cm = static_cast<const T*>(a.C) + p.row * a.sC.b + p.t0 * a.sC.t + g * a.N;
    T* out = static_cast<T*>(a.out) + p.row * a.so.b + p.t0 * a.so.t + d;
    long long chunk = 0;
    if (MODE != kSpanState && a.ckpt)
        chunk = a.s.cu ? slot_base(a.s.cu, p.b, a.s.L, kScanChunk)
                       : p.b * ((a.s.L + kScanChunk - 1) / kScanChunk);

    T ru[K], rd[K], rz[K], rbc[NB];
    auto load_tile = [&](int t0) {
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int t = t0 + k * P + q;
            ru[k] = rd[k] = rz[k] = from_f32<T>(0.f);
            if (t < last) {
                ru[k] = u[t * a.su.t];
                rd[k] = dl[t * a.sdt.t];
                if (MODE != kSpanState && z) rz[k] = z[t * a.sz.t];
            }
        }
#pragma unroll
        for (int k = 0; k < NB; ++k) {
            const int e = k * kWarps * 32 + threadIdx.x, t = t0 + e / (2 * NP), n = e % NP;
            rbc[k] = from_f32<T>(0.f);
            if (e < BC && t < last && (!PAD || n < a.N))
                rbc[k] = (e / NP) & 1 ? Cm[t * a.sC.t + n] : Bm[t * a.sB.t + n];
        }
    };

    float sum_dt = 0.f;
    int buf = 0;
    load_tile(first);
    for (int t0 = first; t0 < last; t0 += kTile, buf ^= 1) {
        float fu[K], fz[K];
#pragma unroll
        for (int k = 0; k < NB; ++k) {
            const int e = k * kWarps * 32 + threadIdx.x;
            if (e < BC) sbc[buf][e] = to_f32(rbc[k]);
        }
#pragma unroll
        for (int k = 0; k < K; ++k) {
            fu[k] = to_f32(ru[k]);
            fz[k] = to_f32(rz[k]);
            float dt = to_f32(rd[k]) + bias;
            if (a.softplus) dt = softplus_f(dt);
            if (t0 + k * P + q >= last) dt = 0.f;
            sum_dt += dt;
            sdt[warp][k * P + q][c] = make_float2(dt, dt * fu[k]);
        }
        __syncthreads();  // B and C of this tile; the other buffer is read no more
        if (t0 + kTile < last) load_tile(t0 + kTile);

        auto tokens = [&](auto full) {
            constexpr bool FULL = decltype(full)::value;
            const int n = FULL ? kTile : last - t0;
#pragma unroll
            for (int k = 0; k < K; ++k) {
                float y[P];
#pragma unroll
                for (int j = 0; j < P; ++j) {
                    const int t = k * P + j;
                    y[j] = 0.f;
                    if (FULL || t < n) {
                        if (MODE != kSpanState && a.ckpt && t % kScanChunk == 0 && live)
                            store_state<PAD>(a.ckpt + (chunk + (t0 + t) / kScanChunk) * hrow + hoff, left, h);
                        const float2 v = sdt[warp][t][c];
                        const float4 b4 = *reinterpret_cast<const float4*>(&sbc[buf][(2 * t) * NP + 4 * q]);
                        const float b[4] = {b4.x, b4.y, b4.z, b4.w};
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            h[i] = fmaf(decay2(v.x * A2[i]), h[i], v.y * b[i]);
                            if (PAD && i >= left) h[i] = 0.f;
                        }
                        if (MODE != kSpanState) {
                            const float4 c4 = *reinterpret_cast<const float4*>(&sbc[buf][(2 * t + 1) * NP + 4 * q]);
                            y[j] = fmaf(c4.x, h[0], c4.y * h[1]) + fmaf(c4.z, h[2], c4.w * h[3]);
                        }
                    }
                }
                if (MODE != kSpanState) {
                    float v = reduce_across<P, CPW>(y, q);
                    const int t = t0 + k * P + q;
                    v = fmaf(Dk, fu[k], v);
                    if (z) v *= silu_f(fz[k]);
                    if (live && (FULL || t < last)) out[t * a.so.t] = from_f32<T>(v);
                }
            }
        };
        if (t0 + kTile <= last) tokens(std::true_type{});
        else tokens(std::false_type{});
        __syncwarp();  // sdt is read no more
    }
    if (MODE == kSpanState) {
#pragma unroll
        for (int w = P / 2; w >= 1; w /= 2) sum_dt += __shfl_xor_sync(0xffffffffu, sum_dt, w * CPW);
        if (live) {
            store_state<PAD>(a.seg_h + p.slot * hrow + hoff, left, h);
            if (q == 0) a.seg_dt[static_cast<long long>(p.slot) * a.dim + d] = sum_dt;
        }
    } else if (a.state_out && page >= 0 && live && last == p.len) {
        store_state<PAD>(a.state_out + page * hrow + hoff, left, h);
    }
}

// One token of each sequence, the state in its page read and written once: 8 N bytes a channel,
// which is what bounds it.  P lanes a channel, as above.
template <typename T, int P, bool PAD>
__global__ void __launch_bounds__(256) scan_step_kernel(const ScanStepArgs a) {
    const long long id = (static_cast<long long>(blockIdx.x) * 256 + threadIdx.x) / P;
    const int q = threadIdx.x % P, b = static_cast<int>(id / a.dim), d = static_cast<int>(id % a.dim);
    const int page = b < a.n_seq ? page_of(a.pages, a.n_pages, b) : -1;
    const bool on = page >= 0;
    float y = 0.f, u = 0.f;
    if (on) {
        const int left = a.N - 4 * q, g = d / (a.dim / a.groups), n = g * a.N + 4 * q;
        float* hp = a.state + (static_cast<long long>(page) * a.dim + d) * a.N + 4 * q;
        float h[4], A[4];
        load_state<PAD>(hp, left, h);
        load_state<PAD>(a.A + static_cast<long long>(d) * a.N + 4 * q, left, A);
        u = to_f32(static_cast<const T*>(a.u)[b * a.su + d]);
        float dt = to_f32(static_cast<const T*>(a.delta)[b * a.sdt + d]) + (a.bias ? a.bias[d] : 0.f);
        if (a.softplus) dt = softplus_f(dt);
        const T* Bm = static_cast<const T*>(a.B) + b * a.sB + n;
        const T* Cm = static_cast<const T*>(a.C) + b * a.sC + n;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (!PAD || i < left) {
                h[i] = fmaf(decay2(dt * (A[i] * kLog2e)), h[i], dt * u * to_f32(Bm[i]));
                y = fmaf(to_f32(Cm[i]), h[i], y);
            }
        }
        store_state<PAD>(hp, left, h);
    }
#pragma unroll
    for (int w = P / 2; w >= 1; w /= 2) y += __shfl_xor_sync(0xffffffffu, y, w);
    if (on && q == 0) {
        y = fmaf(a.D ? a.D[d] : 0.f, u, y);
        if (a.z) y *= silu_f(to_f32(static_cast<const T*>(a.z)[b * a.sz + d]));
        static_cast<T*>(a.out)[b * a.so + d] = from_f32<T>(y);
    }
}

template <typename T, int P, bool PAD>
cudaError_t run(const ScanArgs& a, cudaStream_t s) {
    constexpr int CH = kWarps * 32 / P;
    const int r = a.dim / a.groups, tiles = a.groups * ((r + CH - 1) / CH);
    const unsigned grid = static_cast<unsigned>(static_cast<long long>(a.n_slots) * tiles);
    if (!a.split) {
        scan_kernel<T, P, PAD, kWhole><<<grid, kWarps * 32, 0, s>>>(a);
    } else {
        scan_kernel<T, P, PAD, kSpanState><<<grid, kWarps * 32, 0, s>>>(a);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
        scan_kernel<T, P, PAD, kSpanOut><<<grid, kWarps * 32, 0, s>>>(a);
    }
    return cudaGetLastError();
}
template <typename T, int P, bool PAD>
cudaError_t run_step(const ScanStepArgs& a, cudaStream_t s) {
    const long long n = static_cast<long long>(a.n_seq) * a.dim * P;
    scan_step_kernel<T, P, PAD><<<static_cast<unsigned>((n + 255) / 256), 256, 0, s>>>(a);
    return cudaGetLastError();
}

// Lanes a channel: the fewest that hold N states, 4 each.
template <typename T, class Args, class F>
cudaError_t by_states(const Args& a, F f) {
    if (a.N <= 4) return f(std::integral_constant<int, 1>{});
    if (a.N <= 8) return f(std::integral_constant<int, 2>{});
    if (a.N <= 16) return f(std::integral_constant<int, 4>{});
    if (a.N <= 32) return f(std::integral_constant<int, 8>{});
    return f(std::integral_constant<int, 16>{});
}
template <typename T>
cudaError_t dispatch(const ScanArgs& a, cudaStream_t s) {
    return by_states<T>(a, [&](auto p) {
        constexpr int P = decltype(p)::value;
        return a.N == 4 * P ? run<T, P, false>(a, s) : run<T, P, true>(a, s);
    });
}
template <typename T>
cudaError_t dispatch_step(const ScanStepArgs& a, cudaStream_t s) {
    return by_states<T>(a, [&](auto p) {
        constexpr int P = decltype(p)::value;
        return a.N == 4 * P ? run_step<T, P, false>(a, s) : run_step<T, P, true>(a, s);
    });
}

}  // namespace

int scan_channels(int N) { return kWarps * 32 / (N <= 4 ? 1 : N <= 8 ? 2 : N <= 16 ? 4 : N <= 32 ? 8 : 16); }

cudaError_t launch_scan(const ScanArgs& a, int dtype, cudaStream_t s) {
    return dtype == 0 ? dispatch<float>(a, s) : dispatch<__nv_bfloat16>(a, s);
}

cudaError_t launch_scan_step(const ScanStepArgs& a, int dtype, cudaStream_t s) {
    return dtype == 0 ? dispatch_step<float>(a, s) : dispatch_step<__nv_bfloat16>(a, s);
}

}  // namespace ttt

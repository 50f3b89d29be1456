// causal_conv.cu -- the short causal convolution over tokens, one filter per channel:
//
//   pre[t][d] = bias[d] + sum_w weight[d][w] x[t - (W-1) + w][d],   out = silu(pre) or pre,
//
// for prompts, for single tokens, and its gradient.  Rows before a sequence's first come from its
// page of the state (the W - 1 inputs before it) or are zero.
//
// All three are bound by HBM: the forward reads x and writes out once (2 e bytes a channel and
// token, e the element size) for about 2 W + 6 operations.  A thread owns VEC neighbouring channels
// (16 bytes of them where the alignment allows) and walks down `span` tokens with the last W - 1
// inputs in registers, so each row is read once per block plus W - 1 rows of the block before.
#include "seq_common.cuh"

namespace ttt {
namespace {

constexpr int kThreads = 128;

template <typename T, int W, int VEC>
__global__ void __launch_bounds__(kThreads) conv_kernel(const ConvArgs a) {
    const int d = (blockIdx.y * kThreads + threadIdx.x) * VEC;
    if (d >= a.D) return;
    each_rest_row(a.s, blockIdx.x, gridDim.x, [&](long long r) {
        const float zero[VEC] = {};
        store_vec<VEC>(static_cast<T*>(a.out) + r * a.so.t + d, zero);
    });
    Piece p;
    if (!find_piece(a.s, blockIdx.x, a.span, p)) return;
    const T* x = static_cast<const T*>(a.x) + p.row * a.sx.b + p.t0 * a.sx.t + d;
    T* out = static_cast<T*>(a.out) + p.row * a.so.b + p.t0 * a.so.t + d;
    const int page = page_of(a.pages, a.n_pages, p.b);
    const T* before = a.state_in && page >= 0
        ? static_cast<const T*>(a.state_in) + (static_cast<long long>(page) * (W - 1)) * a.D + d : nullptr;
    float w[W][VEC], bias[VEC], win[W][VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
        bias[i] = a.bias ? a.bias[d + i] : 0.f;
#pragma unroll
        for (int k = 0; k < W; ++k) w[k][i] = a.weight[static_cast<long long>(d + i) * W + k];
    }
    const int first = p.tile * a.span, last = min(first + a.span, p.len);
    // win[0 .. W-2]: the inputs at first - (W-1) .. first - 1
#pragma unroll
    for (int k = 0; k < W - 1; ++k) {
        const int t = first - (W - 1) + k;
        if (t >= 0) {
            load_vec<VEC>(x + t * a.sx.t, win[k]);
        } else if (before) {
            load_vec<VEC>(before + static_cast<long long>(t + W - 1) * a.D, win[k]);
        } else {
#pragma unroll
            for (int i = 0; i < VEC; ++i) win[k][i] = 0.f;
        }
    }
    // The block of a sequence's first tokens also writes its end state: it has read the start state
    // (the same thread, the same channels), so the two may be the same pages.
    if (p.tile == 0 && a.state_out && page >= 0) {
        float keep[W - 1][VEC];
#pragma unroll
        for (int k = 0; k < W - 1; ++k) {
            const int t = p.len - (W - 1) + k;
            if (t >= 0) {
                load_vec<VEC>(x + t * a.sx.t, keep[k]);
            } else {
#pragma unroll
                for (int j = 0; j < W - 1; ++j)
                    if (j == t + W - 1)
#pragma unroll
                        for (int i = 0; i < VEC; ++i) keep[k][i] = win[j][i];
            }
        }
        T* after = static_cast<T*>(a.state_out) + (static_cast<long long>(page) * (W - 1)) * a.D + d;
#pragma unroll
        for (int k = 0; k < W - 1; ++k) store_vec<VEC>(after + static_cast<long long>(k) * a.D, keep[k]);
    }
    constexpr int U = 4;  // rows loaded ahead of their use
    for (int t = first; t < last; t += U) {
        float rows[U][VEC];
#pragma unroll
        for (int r = 0; r < U; ++r)
            if (t + r < last) load_vec<VEC>(x + (t + r) * a.sx.t, rows[r]);
#pragma unroll
        for (int r = 0; r < U; ++r) {
            if (t + r < last) {
                float y[VEC];
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    win[W - 1][i] = rows[r][i];
                    float acc = bias[i];
#pragma unroll
                    for (int k = 0; k < W; ++k) acc = fmaf(w[k][i], win[k][i], acc);
                    y[i] = a.silu ? silu_f(acc) : acc;
#pragma unroll
                    for (int k = 0; k < W - 1; ++k) win[k][i] = win[k + 1][i];
                }
                store_vec<VEC>(out + (t + r) * a.so.t, y);
            }
        }
    }
}

// One token of each sequence: the state's window moves on by one row, in place.
template <typename T, int W, int VEC>
__global__ void __launch_bounds__(kThreads) conv_step_kernel(const ConvArgs a) {
    const int per = (a.D + VEC - 1) / VEC;
    const long long i = static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x;
    const int b = static_cast<int>(i / per), d = static_cast<int>(i % per) * VEC;
    if (b >= a.s.n_seq) return;
    const int page = page_of(a.pages, a.n_pages, b);
    if (page < 0) {
        const float zero[VEC] = {};
        store_vec<VEC>(static_cast<T*>(a.out) + b * a.so.b + d, zero);
        return;
    }
    T* state = static_cast<T*>(a.state_out) + (static_cast<long long>(page) * (W - 1)) * a.D + d;
    float win[W][VEC], y[VEC];
#pragma unroll
    for (int k = 0; k < W - 1; ++k) load_vec<VEC>(state + static_cast<long long>(k) * a.D, win[k]);
    load_vec<VEC>(static_cast<const T*>(a.x) + b * a.sx.b + d, win[W - 1]);
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
        float acc = a.bias ? a.bias[d + j] : 0.f;
#pragma unroll
        for (int k = 0; k < W; ++k) acc = fmaf(a.weight[static_cast<long long>(d + j) * W + k], win[k][j], acc);
        y[j] = a.silu ? silu_f(acc) : acc;
    }
#pragma unroll
    for (int k = 0; k < W - 1; ++k) store_vec<VEC>(state + static_cast<long long>(k) * a.D, win[k + 1]);
    store_vec<VEC>(static_cast<T*>(a.out) + b * a.so.b + d, y);
}

// Gradients.  With dpre = d_out * silu'(pre) (pre is computed again from x):
//   dx[t] = sum_w weight[w] dpre[t + W-1 - w],  d_weight[w] = sum_t dpre[t] x[t - (W-1) + w],
//   d_bias = sum_t dpre[t];  rows past the sequence have dpre = 0, and dx at the rows before it is
//   the gradient of its start state.  A thread walks down the rows of its span and W - 1 rows more
//   (whose dpre the span's last rows need), with the last W inputs and the last W dpre in registers.
// d_weight and d_bias are sums over every row: each block writes its own, and a second kernel adds
// the blocks' in a fixed order.
template <typename T, int W, int VEC>
__global__ void __launch_bounds__(kThreads) conv_bwd_kernel(const ConvBwdArgs a) {
    const int d = (blockIdx.y * kThreads + threadIdx.x) * VEC;
    if (d >= a.D) return;
    each_rest_row(a.s, blockIdx.x, gridDim.x, [&](long long r) {
        const float zero[VEC] = {};
        store_vec<VEC>(static_cast<T*>(a.dx) + r * a.D + d, zero);
    });
    float* part = a.part + static_cast<long long>(blockIdx.x) * (W + 1) * a.D + d;
    float gw[W][VEC], gb[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
        gb[i] = 0.f;
#pragma unroll
        for (int k = 0; k < W; ++k) gw[k][i] = 0.f;
    }
    Piece p;
    if (find_piece(a.s, blockIdx.x, a.span, p)) {
        const T* x = static_cast<const T*>(a.x) + p.row * a.sx.b + p.t0 * a.sx.t + d;
        const T* dy = static_cast<const T*>(a.d_out) + p.row * a.sd.b + p.t0 * a.sd.t + d;
        T* dx = static_cast<T*>(a.dx) + (p.row * a.s.L + p.t0) * a.D + d;
        const long long st = static_cast<long long>(p.b) * (W - 1) * a.D + d;
        const T* before = a.state_in ? static_cast<const T*>(a.state_in) + st : nullptr;
        const T* after = a.d_state_out ? static_cast<const T*>(a.d_state_out) + st : nullptr;
        T* dbefore = a.d_state_in ? static_cast<T*>(a.d_state_in) + st : nullptr;
        float w[W][VEC], bias[VEC], win[W][VEC], dp[W][VEC];
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            bias[i] = a.bias ? a.bias[d + i] : 0.f;
#pragma unroll
            for (int k = 0; k < W; ++k) {
                w[k][i] = a.weight[static_cast<long long>(d + i) * W + k];
                dp[k][i] = 0.f;
            }
        }
        const int first = p.tile * a.span, last = min(first + a.span, p.len);
#pragma unroll
        for (int k = 0; k < W - 1; ++k) {
            const int t = first - (W - 1) + k;
            if (t >= 0) {
                load_vec<VEC>(x + t * a.sx.t, win[k]);
            } else if (before) {
                load_vec<VEC>(before + static_cast<long long>(t + W - 1) * a.D, win[k]);
            } else {
#pragma unroll
                for (int i = 0; i < VEC; ++i) win[k][i] = 0.f;
            }
        }
        // row r: dpre[r] joins dp[W-1]; then dx[r - (W-1)] = sum_w weight[w] dpre[r - w]
        constexpr int U = 4;
        const int stop = last + W - 1;
        for (int t = first; t < stop; t += U) {
            float xr[U][VEC], dr[U][VEC];
#pragma unroll
            for (int r = 0; r < U; ++r)
                if (t + r < stop && t + r < p.len) {
                    load_vec<VEC>(x + (t + r) * a.sx.t, xr[r]);
                    load_vec<VEC>(dy + (t + r) * a.sd.t, dr[r]);
                }
#pragma unroll
            for (int r = 0; r < U; ++r) {
                const int row = t + r;
                if (row < stop) {
                    float g[VEC];
#pragma unroll
                    for (int i = 0; i < VEC; ++i) {
                        float dpre = 0.f;
                        if (row < p.len) {
                            win[W - 1][i] = xr[r][i];
                            dpre = dr[r][i];
                            if (a.silu) {
                                float pre = bias[i];
#pragma unroll
                                for (int k = 0; k < W; ++k) pre = fmaf(w[k][i], win[k][i], pre);
                                dpre *= silu_grad_f(pre, sigmoid_f(pre));
                            }
                            if (row < last) {
                                gb[i] += dpre;
#pragma unroll
                                for (int k = 0; k < W; ++k) gw[k][i] = fmaf(dpre, win[k][i], gw[k][i]);
                            }
#pragma unroll
                            for (int k = 0; k < W - 1; ++k) win[k][i] = win[k + 1][i];
                        }
                        dp[W - 1][i] = dpre;
                        g[i] = 0.f;
#pragma unroll
                        for (int k = 0; k < W; ++k) g[i] = fmaf(w[k][i], dp[W - 1 - k][i], g[i]);
#pragma unroll
                        for (int k = 0; k < W - 1; ++k) dp[k][i] = dp[k + 1][i];
                    }
                    const int at = row - (W - 1);  // the row whose gradient is complete
                    if (after && at >= p.len - (W - 1) && (at >= first || at < 0)) {
                        float e[VEC];
                        load_vec<VEC>(after + static_cast<long long>(at - (p.len - (W - 1))) * a.D, e);
#pragma unroll
                        for (int i = 0; i < VEC; ++i) g[i] += e[i];
                    }
                    if (at >= first && at < last) store_vec<VEC>(dx + static_cast<long long>(at) * a.D, g);
                    else if (at < 0 && dbefore) store_vec<VEC>(dbefore + static_cast<long long>(at + W - 1) * a.D, g);
                }
            }
        }
    }
#pragma unroll
    for (int k = 0; k < W; ++k) store_vec<VEC>(part + static_cast<long long>(k) * a.D, gw[k]);
    store_vec<VEC>(part + static_cast<long long>(W) * a.D, gb);
}

// d_weight[d][w] and d_bias[d]: the sum over the blocks' shares, 8 runs of them side by side.
__global__ void __launch_bounds__(256) conv_bwd_sum_kernel(const ConvBwdArgs a) {
    __shared__ float sh[8][32];
    const int col = blockIdx.x * 32 + (threadIdx.x & 31), run = threadIdx.x >> 5;
    const int cols = (a.W + 1) * a.D;
    float s = 0.f;
    if (col < cols)
        for (int k = run; k < a.n_slots; k += 8) s += a.part[static_cast<long long>(k) * cols + col];
    sh[run][threadIdx.x & 31] = s;
    __syncthreads();
    if (run == 0 && col < cols) {
#pragma unroll
        for (int k = 1; k < 8; ++k) s += sh[k][threadIdx.x];
        const int w = col / a.D, d = col % a.D;
        if (w < a.W) a.d_weight[static_cast<long long>(d) * a.W + w] = s;
        else if (a.d_bias) a.d_bias[d] = s;
    }
}

long long slots(const SeqShape& s, int span) {
    return s.cu ? s.L / span + s.n_seq : s.n_seq * (s.L > 0 ? (s.L + span - 1) / span : 1);
}

bool rows_fit(const void* p, RowStride r, size_t esz, size_t bytes) {
    return reinterpret_cast<uintptr_t>(p) % bytes == 0 && (r.b * esz) % bytes == 0 && (r.t * esz) % bytes == 0;
}

template <typename T, int W, int VEC>
cudaError_t fwd(const ConvArgs& a, cudaStream_t s) {
    const int gy = (a.D + kThreads * VEC - 1) / (kThreads * VEC);
    conv_kernel<T, W, VEC><<<dim3(static_cast<unsigned>(slots(a.s, a.span)), gy), kThreads, 0, s>>>(a);
    return cudaGetLastError();
}
template <typename T, int W, int VEC>
cudaError_t step(const ConvArgs& a, cudaStream_t s) {
    const long long n = static_cast<long long>(a.s.n_seq) * ((a.D + VEC - 1) / VEC);
    conv_step_kernel<T, W, VEC><<<static_cast<unsigned>((n + kThreads - 1) / kThreads), kThreads, 0, s>>>(a);
    return cudaGetLastError();
}
template <typename T, int W, int VEC>
cudaError_t bwd(const ConvBwdArgs& a, cudaStream_t s) {
    const int gy = (a.D + kThreads * VEC - 1) / (kThreads * VEC);
    conv_bwd_kernel<T, W, VEC><<<dim3(a.n_slots, gy), kThreads, 0, s>>>(a);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    conv_bwd_sum_kernel<<<((a.W + 1) * a.D + 31) / 32, 256, 0, s>>>(a);
    return cudaGetLastError();
}

#define TTT_CONV_WIDTH(F, T, VEC)            \
    switch (a.W) {                           \
        case 2: return F<T, 2, VEC>(a, s);   \
        case 3: return F<T, 3, VEC>(a, s);   \
        case 4: return F<T, 4, VEC>(a, s);   \
        default: return cudaErrorInvalidValue; \
    }

}  // namespace

// 16 bytes of channels a thread where every row starts on such a boundary, one channel otherwise.
static bool wide(const ConvArgs& a, size_t esz) {
    const int v = static_cast<int>(16 / esz);
    const RowStride st{a.D, a.D};
    return a.D % v == 0 && rows_fit(a.x, a.sx, esz, 16) && rows_fit(a.out, a.so, esz, 16) &&
           rows_fit(a.state_in, st, esz, 16) && rows_fit(a.state_out, st, esz, 16);
}

cudaError_t launch_conv(const ConvArgs& args, int dtype, cudaStream_t s) {
    ConvArgs a = args;
    const bool v = wide(a, dtype == 0 ? 4 : 2);
    a.span = 32;
    if (dtype == 0) {
        if (v) { TTT_CONV_WIDTH(fwd, float, 4) }
        TTT_CONV_WIDTH(fwd, float, 1)
    }
    if (v) { TTT_CONV_WIDTH(fwd, __nv_bfloat16, 8) }
    TTT_CONV_WIDTH(fwd, __nv_bfloat16, 1)
}

cudaError_t launch_conv_step(const ConvArgs& a, int dtype, cudaStream_t s) {
    const bool v = wide(a, dtype == 0 ? 4 : 2);
    if (dtype == 0) {
        if (v) { TTT_CONV_WIDTH(step, float, 4) }
        TTT_CONV_WIDTH(step, float, 1)
    }
    if (v) { TTT_CONV_WIDTH(step, __nv_bfloat16, 8) }
    TTT_CONV_WIDTH(step, __nv_bfloat16, 1)
}

int conv_bwd_span(int n_seq, long long L, bool packed, int D, int dtype) { return 32; }

cudaError_t launch_conv_bwd(const ConvBwdArgs& a, int dtype, cudaStream_t s) {
    const size_t esz = dtype == 0 ? 4 : 2;
    const RowStride st{a.D, a.D};
    const int v = 4;  // channels a thread: 8 or 16 bytes, and registers enough for two windows
    const bool fits = a.D % v == 0 && rows_fit(a.x, a.sx, esz, v * esz) && rows_fit(a.d_out, a.sd, esz, v * esz) &&
                      rows_fit(a.dx, st, esz, v * esz) && rows_fit(a.state_in, st, esz, v * esz) &&
                      rows_fit(a.d_state_out, st, esz, v * esz) && rows_fit(a.d_state_in, st, esz, v * esz);
    if (dtype == 0) {
        if (fits) { TTT_CONV_WIDTH(bwd, float, 4) }
        TTT_CONV_WIDTH(bwd, float, 1)
    }
    if (fits) { TTT_CONV_WIDTH(bwd, __nv_bfloat16, 4) }
    TTT_CONV_WIDTH(bwd, __nv_bfloat16, 1)
}

}  // namespace ttt

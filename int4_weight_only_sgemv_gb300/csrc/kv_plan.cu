// Block tables and slot maps of one step from the requests' lengths.
//
// Every CTA scans all requests by itself (three counts each), so no CTA waits for another; the outputs are then
// spread over the whole grid. Nothing that is read is written: pages that change hands are found by their rank
// among the given-up and the handed-out pages, not by the order in which threads reach the stack.
#include <algorithm>

#include "kv_common.cuh"

namespace sgemv {

namespace {

constexpr int kPlanThreads = 512;

struct PlanParams {
    const int32_t* len;
    const int32_t* keep;  // nullable
    const int32_t* add;
    int32_t* table;
    int64_t table_stride;
    int32_t* free;
    const int32_t* free_count;
    int32_t* len_out;
    int32_t* free_count_out;
    int32_t* q_start;
    int64_t* slots;
    int32_t* pos;
    int32_t* status;
    int n_req, page, n_pages, table_cols, n_slots;
};

// What one request (or a run of them) adds, gives up and is handed.
struct Counts {
    int64_t add, gone, come;
};

struct Request {
    int len, keep, add, held, need;  // pages held before and needed after
};

__device__ __forceinline__ Request request(const PlanParams& p, int r) {
    Request q;
    q.len = p.len[r];
    q.keep = p.keep != nullptr ? p.keep[r] : q.len;
    q.add = p.add[r];
    q.held = static_cast<int>((static_cast<int64_t>(q.len) + p.page - 1) / p.page);
    q.need = static_cast<int>((static_cast<int64_t>(q.keep) + q.add + p.page - 1) / p.page);
    return q;
}

__device__ __forceinline__ Counts counts(const Request& q) {
    return {q.add, q.held > q.need ? q.held - q.need : 0, q.need > q.held ? q.need - q.held : 0};
}

// The last i in [0, n) with a[i] <= x (a[0] <= x).
__device__ __forceinline__ int find(const int64_t* a, int n, int64_t x) {
    int lo = 0, hi = n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (a[mid] <= x) lo = mid; else hi = mid - 1;
    }
    return lo;
}

__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const PlanParams p) {
    __shared__ int64_t s_add[kPlanThreads], s_gone[kPlanThreads], s_come[kPlanThreads];
    __shared__ int64_t s_warp[3][kPlanThreads / 32];
    __shared__ int s_err;
    pdl_launch_dependents();
    pdl_wait();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    // thread t has the requests [t * run, (t + 1) * run)
    const int run = (p.n_req + kPlanThreads - 1) / kPlanThreads;
    if (tid == 0) s_err = 0;
    __syncthreads();
    Counts sum = {0, 0, 0};
    const int r0 = static_cast<int>(min(static_cast<int64_t>(tid) * run, static_cast<int64_t>(p.n_req)));
    const int r1 = min(r0 + run, p.n_req);
    for (int r = r0; r < r1; ++r) {
        const Request q = request(p, r);
        if (q.len < 0 || q.keep < 0 || q.keep > q.len || q.add < 0 || static_cast<int64_t>(q.keep) + q.add > INT32_MAX)
            s_err = SGEMV_ERR_ARG;
        else if (max(q.held, q.need) > p.table_cols)
            atomicCAS(&s_err, 0, SGEMV_ERR_SHAPE);
        const Counts c = counts(q);
        sum.add += c.add, sum.gone += c.gone, sum.come += c.come;
    }
    // exclusive prefix sums over the threads
    Counts incl = sum;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int64_t a = __shfl_up_sync(0xFFFFFFFFu, incl.add, d), g = __shfl_up_sync(0xFFFFFFFFu, incl.gone, d),
                      c = __shfl_up_sync(0xFFFFFFFFu, incl.come, d);
        if (lane >= d) incl.add += a, incl.gone += g, incl.come += c;
    }
    if (lane == 31) s_warp[0][warp] = incl.add, s_warp[1][warp] = incl.gone, s_warp[2][warp] = incl.come;
    __syncthreads();
    Counts before = {0, 0, 0}, all = {0, 0, 0};
    for (int w = 0; w < kPlanThreads / 32; ++w) {
        if (w < warp) before.add += s_warp[0][w], before.gone += s_warp[1][w], before.come += s_warp[2][w];
        all.add += s_warp[0][w], all.gone += s_warp[1][w], all.come += s_warp[2][w];
    }
    before.add += incl.add - sum.add, before.gone += incl.gone - sum.gone, before.come += incl.come - sum.come;
    s_add[tid] = before.add, s_gone[tid] = before.gone, s_come[tid] = before.come;
    __syncthreads();
    const int n_free = *p.free_count;
    int err = s_err;
    if (err == 0 && (all.add > p.n_slots || n_free < 0 || n_free > p.n_pages)) err = SGEMV_ERR_ARG;
    if (err == 0 && (all.come - all.gone > n_free || all.gone - all.come > p.n_pages - n_free)) err = SGEMV_ERR_SHAPE;
    const bool ok = err == 0;
    if (!ok && blockIdx.x == 0 && tid == 0) report(p.status, err);

    // per request: thread t's run by CTA t % grid
    if (tid % gridDim.x == blockIdx.x) {
        int64_t at = before.add;
        for (int r = r0; r < r1; ++r) {
            const Request q = request(p, r);
            p.q_start[r] = ok ? static_cast<int32_t>(at) : 0;
            p.len_out[r] = ok ? q.keep + q.add : q.len;
            at += q.add;
        }
    }
    if (blockIdx.x == 0 && tid == 0) {
        p.q_start[p.n_req] = ok ? static_cast<int32_t>(all.add) : 0;
        *p.free_count_out = ok ? static_cast<int32_t>(n_free + all.gone - all.come) : n_free;
    }

    const int64_t first = static_cast<int64_t>(blockIdx.x) * kPlanThreads + tid;
    const int64_t stride = static_cast<int64_t>(gridDim.x) * kPlanThreads;
    const int n_run = run > 0 ? min(kPlanThreads, (p.n_req + run - 1) / run) : 0;

    // the i-th page that a request gives up
    const auto given = [&](int64_t i) {
        const int t = find(s_gone, n_run, i);
        int64_t at = s_gone[t];
        for (int r = t * run;; ++r) {
            const Request q = request(p, r);
            const int64_t n = counts(q).gone;
            if (i < at + n) return p.table[r * p.table_stride + q.need + (i - at)];
            at += n;
        }
    };
    // the i-th page that a request is handed
    const auto handed = [&](int64_t i) {
        return i < all.gone ? given(i) : p.free[n_free - 1 - (i - all.gone)];
    };
    if (ok) {
        for (int64_t i = first; i < all.come; i += stride) {
            const int t = find(s_come, n_run, i);
            int64_t at = s_come[t];
            int r = t * run;
            Request q = request(p, r);
            while (i >= at + counts(q).come) {
                at += counts(q).come;
                q = request(p, ++r);
            }
            p.table[r * p.table_stride + q.held + (i - at)] = handed(i);
        }
        for (int64_t i = all.come + first; i < all.gone; i += stride) p.free[n_free + i - all.come] = given(i);
    }
    for (int64_t i = first; i < p.n_slots; i += stride) {
        int64_t slot = -1;
        int pos = -1;
        if (ok && i < all.add) {
            const int t = find(s_add, n_run, i);
            int64_t at = s_add[t], come = s_come[t];
            int r = t * run;
            Request q = request(p, r);
            while (i >= at + q.add) {
                at += q.add, come += counts(q).come;
                q = request(p, ++r);
            }
            pos = q.keep + static_cast<int>(i - at);
            const int b = pos / p.page;
            const int id = b < q.held ? p.table[r * p.table_stride + b] : handed(come + (b - q.held));
            if (id >= 0 && id < p.n_pages) slot = static_cast<int64_t>(id) * p.page + pos % p.page;
            else report(p.status, SGEMV_ERR_ARG);
        }
        p.slots[i] = slot;
        p.pos[i] = pos;
    }
}

}  // namespace

}  // namespace sgemv

using namespace sgemv;

extern "C" int sgemv_kv_plan(int n_req, int page, int n_pages, const int32_t* len_dev, const int32_t* keep_dev,
                             const int32_t* add_dev, int32_t* table_dev, int table_cols, int64_t table_stride,
                             int32_t* free_dev, const int32_t* free_count_dev, int32_t* len_out_dev,
                             int32_t* free_count_out_dev, int32_t* q_start_dev, int64_t* slots_dev, int32_t* pos_dev,
                             int n_slots, int32_t* status_dev, void* stream) {
    if (n_req < 0 || n_slots < 0 || table_cols < 1 || table_stride < table_cols || n_pages < 1) return SGEMV_ERR_ARG;
    if (page != 16 && page != 32 && page != 64 && page != 128 && page != 256) return SGEMV_ERR_SHAPE;
    const void* must[] = {free_dev, free_count_dev, free_count_out_dev, q_start_dev};
    for (const void* q : must)
        if (q == nullptr) return SGEMV_ERR_ARG;
    if (n_req > 0 && (len_dev == nullptr || add_dev == nullptr || table_dev == nullptr || len_out_dev == nullptr))
        return SGEMV_ERR_ARG;
    if (n_slots > 0 && (slots_dev == nullptr || pos_dev == nullptr)) return SGEMV_ERR_ARG;
    const void* ptrs[] = {len_dev,            keep_dev,    add_dev, table_dev, free_dev, free_count_dev, len_out_dev,
                          free_count_out_dev, q_start_dev, pos_dev, status_dev};
    for (const void* q : ptrs)
        if (!is_aligned(q, 4)) return SGEMV_ERR_ALIGN;
    if (!is_aligned(slots_dev, 8)) return SGEMV_ERR_ALIGN;
    if (free_count_dev == free_count_out_dev || (n_req > 0 && (len_dev == len_out_dev || keep_dev == len_out_dev ||
                                                               add_dev == len_out_dev)))
        return SGEMV_ERR_ARG;
    DeviceInfo di;
    const int rc = device_info(&di);
    if (rc != SGEMV_OK) return rc;
    PlanParams p;
    p.len = len_dev;
    p.keep = keep_dev;
    p.add = add_dev;
    p.table = table_dev;
    p.table_stride = table_stride;
    p.free = free_dev;
    p.free_count = free_count_dev;
    p.len_out = len_out_dev;
    p.free_count_out = free_count_out_dev;
    p.q_start = q_start_dev;
    p.slots = slots_dev;
    p.pos = pos_dev;
    p.status = status_dev;
    p.n_req = n_req;
    p.page = page;
    p.n_pages = n_pages;
    p.table_cols = table_cols;
    p.n_slots = n_slots;
    const int grid = std::max(1, std::min(di.sm_count, (std::max(n_req, n_slots) + kPlanThreads - 1) / kPlanThreads));
    const cudaError_t e = launch_pdl(plan_kernel, dim3(grid), dim3(kPlanThreads), 0, static_cast<cudaStream_t>(stream), p);
    return e == cudaSuccess ? SGEMV_OK : SGEMV_ERR_CUDA;
}

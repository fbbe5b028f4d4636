// Block tables and slot maps of one step from the requests' lengths.
//
// Every CTA scans all requests by itself (three counts each, prefix sums in shared memory), so no CTA waits for another; the
// outputs are then spread over the whole grid, a token or a page a thread, which finds its request by a binary search.
// Nothing that is read is written: pages that change hands are found by their rank among the given-up and the handed-out
// pages, not by the order in which threads reach the stack.
//
// Bound by latency: a launch, two rounds of dependent loads and the scan. With the prefix sums of runs of requests alone, and
// a walk through global memory from there, 4096 requests took 27 us; so they take 12.8, and 64 requests 4.4 on the GPU (8.5 with the
// host's call).
#include <algorithm>

#include "kv_common.cuh"

namespace sgemv {

namespace {

constexpr int kPlanMaxReq = 16384;  // three prefix sums of so many requests fit in shared memory
constexpr int kPlanMax = 1 << 30;   // slots and pages: an index and a grid's stride past it stay in 32 bits

// Place of request r in shared memory: one word more every 32, so that threads with 8 (or 4, 16) requests each hit all banks.
__host__ __device__ constexpr int padded(int r) { return r + (r >> 5); }

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
    int n_req, log2_page, n_pages, table_cols, n_slots;
};

// Pages of n tokens.
__device__ __forceinline__ int pages_of(const PlanParams& p, int64_t n) {
    return static_cast<int>((n + (1 << p.log2_page) - 1) >> p.log2_page);
}

// The last r in [0, n) with a[r] <= x (a[0] <= x): of requests with the same prefix sum the last, which is the one that is not empty.
__device__ __forceinline__ int find(const int32_t* a, int n, int x) {
    int lo = 0, hi = n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (a[padded(mid)] <= x) lo = mid; else hi = mid - 1;
    }
    return lo;
}

template <int kPlanThreads>
__global__ void __launch_bounds__(kPlanThreads, 1) plan_kernel(const PlanParams p) {
    extern __shared__ int32_t s_sums[];  // of tokens, of pages given up, of pages handed out, before each request
    int32_t* const s_add = s_sums;
    int32_t* const s_gone = s_add + padded(p.n_req);
    int32_t* const s_come = s_gone + padded(p.n_req);
    __shared__ int64_t s_warp[3][kPlanThreads / 32];
    __shared__ int s_err;
    pdl_launch_dependents();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid == 0) s_err = 0;
    __syncthreads();
    pdl_wait();
    const int n_free = *p.free_count;
#pragma unroll 4
    for (int r = tid; r < p.n_req; r += kPlanThreads) {
        const int len = p.len[r], keep = p.keep != nullptr ? p.keep[r] : len, add = p.add[r];
        const int64_t total = static_cast<int64_t>(keep) + add;
        const int held = pages_of(p, len), need = pages_of(p, total);
        if (len < 0 || keep < 0 || keep > len || add < 0 || total > INT32_MAX) s_err = SGEMV_ERR_ARG;
        else if (max(held, need) > p.table_cols) atomicCAS(&s_err, 0, SGEMV_ERR_SHAPE);
        s_add[padded(r)] = add;
        s_gone[padded(r)] = max(held - need, 0);
        s_come[padded(r)] = max(need - held, 0);
    }
    __syncthreads();
    // exclusive prefix sums: thread t has the requests [t * run, (t + 1) * run)
    const int run = (p.n_req + kPlanThreads - 1) / kPlanThreads;
    const int r0 = min(tid * run, p.n_req), r1 = min(r0 + run, p.n_req);
    int64_t sum[3] = {0, 0, 0}, incl[3];
    for (int r = r0; r < r1; ++r) sum[0] += s_add[padded(r)], sum[1] += s_gone[padded(r)], sum[2] += s_come[padded(r)];
#pragma unroll
    for (int x = 0; x < 3; ++x) incl[x] = sum[x];
#pragma unroll
    for (int d = 1; d < 32; d <<= 1)
#pragma unroll
        for (int x = 0; x < 3; ++x) {
            const int64_t o = __shfl_up_sync(0xFFFFFFFFu, incl[x], d);
            if (lane >= d) incl[x] += o;
        }
    if (lane == 31)
        for (int x = 0; x < 3; ++x) s_warp[x][warp] = incl[x];
    __syncthreads();
    int64_t before[3], all[3] = {0, 0, 0};
#pragma unroll
    for (int x = 0; x < 3; ++x) {
        before[x] = incl[x] - sum[x];
#pragma unroll
        for (int w = 0; w < kPlanThreads / 32; ++w) {
            if (w < warp) before[x] += s_warp[x][w];
            all[x] += s_warp[x][w];
        }
    }
    int32_t at[3] = {static_cast<int32_t>(before[0]), static_cast<int32_t>(before[1]), static_cast<int32_t>(before[2])};
    for (int r = r0; r < r1; ++r) {
        const int i = padded(r);
        const int32_t a = s_add[i], g = s_gone[i], c = s_come[i];
        s_add[i] = at[0], s_gone[i] = at[1], s_come[i] = at[2];
        at[0] += a, at[1] += g, at[2] += c;
    }
    __syncthreads();
    int err = s_err;
    if (err == 0 && (all[0] > p.n_slots || n_free < 0 || n_free > p.n_pages)) err = SGEMV_ERR_ARG;
    // (no more pages can change hands than there are: counts and indexes stay in 32 bits)
    if (err == 0 && (all[1] > p.n_pages || all[2] > p.n_pages)) err = SGEMV_ERR_SHAPE;
    if (err == 0 && (all[2] - all[1] > n_free || all[1] - all[2] > p.n_pages - n_free)) err = SGEMV_ERR_SHAPE;
    const bool ok = err == 0;
    const int tokens = ok ? static_cast<int>(all[0]) : 0, gone = ok ? static_cast<int>(all[1]) : 0, come = ok ? static_cast<int>(all[2]) : 0;

    const int first = blockIdx.x * kPlanThreads + tid, stride = gridDim.x * kPlanThreads;
    if (first == 0) {
        if (!ok) report(p.status, err);
        p.q_start[p.n_req] = tokens;
        *p.free_count_out = n_free + gone - come;
    }
    for (int r = first; r < p.n_req; r += stride) {
        const int len = p.len[r];
        p.q_start[r] = ok ? s_add[padded(r)] : 0;
        p.len_out[r] = ok ? (p.keep != nullptr ? p.keep[r] : len) + p.add[r] : len;
    }
    // the i-th page that a request gives up: block need + (i - its first) of it
    const auto given = [&](int i) {
        const int r = find(s_gone, p.n_req, i);
        const int need = pages_of(p, static_cast<int64_t>(p.keep != nullptr ? p.keep[r] : p.len[r]) + p.add[r]);
        return p.table[r * p.table_stride + need + (i - s_gone[padded(r)])];
    };
    // the i-th page that a request is handed
    const auto handed = [&](int i) { return i < gone ? given(i) : p.free[n_free - 1 - (i - gone)]; };
    for (int i = first; i < come; i += stride) {
        const int r = find(s_come, p.n_req, i);
        p.table[r * p.table_stride + pages_of(p, p.len[r]) + (i - s_come[padded(r)])] = handed(i);
    }
    for (int i = come + first; i < gone; i += stride) {
        const int id = given(i);
        if (id < 0 || id >= p.n_pages) report(p.status, SGEMV_ERR_ARG);  // (one that is handed on shows in its tokens' slots)
        p.free[n_free + i - come] = id;
    }
#pragma unroll 2
    for (int i = first; i < p.n_slots; i += stride) {
        int64_t slot = -1;
        int pos = -1;
        if (i < tokens) {
            const int r = find(s_add, p.n_req, i);
            const int len = p.len[r];
            pos = (p.keep != nullptr ? p.keep[r] : len) + (i - s_add[padded(r)]);
            const int b = pos >> p.log2_page, held = pages_of(p, len);
            const int id = b < held ? p.table[r * p.table_stride + b] : handed(s_come[padded(r)] + (b - held));
            if (id >= 0 && id < p.n_pages) slot = (static_cast<int64_t>(id) << p.log2_page) + (pos & ((1 << p.log2_page) - 1));
            else report(p.status, SGEMV_ERR_ARG);
        }
        p.slots[i] = slot;
        p.pos[i] = pos;
    }
}

template <int kPlanThreads>
int launch_plan(const PlanParams& p, const DeviceInfo& di, cudaStream_t s) {
    const uint32_t smem = static_cast<uint32_t>(padded(p.n_req)) * 12;
    if (smem > 44 * 1024) {  // the kernel has some of its own
        static std::atomic<int> attr_set[64];  // per device: dynamic shared memory already enabled
        int dev = 0;
        if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return SGEMV_ERR_CUDA;
        if (attr_set[dev].load() == 0) {
            if (cudaFuncSetAttribute(plan_kernel<kPlanThreads>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     padded(kPlanMaxReq) * 12) != cudaSuccess)
                return SGEMV_ERR_CUDA;
            attr_set[dev].store(1);
        }
    }
    // a token a thread, up to a CTA an SM
    const int grid = std::max(1, std::min(di.sm_count, (std::max(p.n_req, p.n_slots) + kPlanThreads - 1) / kPlanThreads));
    return launch_pdl(plan_kernel<kPlanThreads>, dim3(grid), dim3(kPlanThreads), smem, s, p) == cudaSuccess ? SGEMV_OK : SGEMV_ERR_CUDA;
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
    if (n_req > kPlanMaxReq || n_slots > kPlanMax || n_pages > kPlanMax) return SGEMV_ERR_SHAPE;
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
    const uint64_t per_req = 4ull * n_req;
    const Bytes written[] = {{len_out_dev, per_req}, {free_count_out_dev, 4}, {q_start_dev, per_req + 4}, {slots_dev, 8ull * n_slots},
                             {pos_dev, 4ull * n_slots}, {free_dev, 4ull * n_pages}, {status_dev, 4}};
    const Bytes read[] = {{len_dev, per_req}, {keep_dev, per_req}, {add_dev, per_req}, {free_count_dev, 4}};
    if (!apart(written, read)) return SGEMV_ERR_ARG;
    const Bytes row(table_dev, 4ull * table_cols);  // the table's rows are written too
    for (const Bytes& b : written)
        if (rows_meet(row, n_req, 4ull * table_stride, b)) return SGEMV_ERR_ARG;
    for (const Bytes& b : read)
        if (rows_meet(row, n_req, 4ull * table_stride, b)) return SGEMV_ERR_ARG;
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
    p.log2_page = 0;
    while ((1 << p.log2_page) < page) ++p.log2_page;
    p.n_pages = n_pages;
    p.table_cols = table_cols;
    p.n_slots = n_slots;
    // a decode step of up to 256 requests is all latency: fewer warps to bring together; more work needs them
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    return n_req <= 256 && n_slots <= 4096 ? launch_plan<256>(p, di, st) : launch_plan<1024>(p, di, st);
}

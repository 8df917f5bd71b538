// C-ABI entry points of the rotary positions and the paged cache: argument
// validation and workspace layout.

#include "paged_cache.cuh"

namespace {

using namespace tc;

constexpr size_t kAlign = 256;
size_t round_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }
bool aligned(const void *p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
size_t elem(tc_dtype d) { return d == TC_BF16 ? 2 : 4; }
bool valid_dtype(tc_dtype d) { return d == TC_F32 || d == TC_BF16; }

bool non_negative(const int64_t *s) { return s[0] >= 0 && s[1] >= 0 && s[2] >= 0; }

// Elements spanned by dimensions of `size` with `stride`, 0 when one is empty.
int64_t extent(const int64_t *stride, const int64_t *size, int64_t d) {
    int64_t e = d;
    for (int i = 0; i < 3; ++i) {
        if (size[i] == 0) return 0;
        e += (size[i] - 1) * stride[i];
    }
    return e;
}

// Whether rows of d elements at these strides cannot overlap one another:
// sorted by stride, each stride is at least the extent below it.
bool nested(const int64_t *stride, const int64_t *size, int64_t d) {
    if (size[0] == 0 || size[1] == 0 || size[2] == 0) return true;
    int order[3] = {0, 1, 2};
    for (int i = 0; i < 3; ++i)
        for (int j = i + 1; j < 3; ++j)
            if (stride[order[j]] < stride[order[i]]) {
                const int t = order[i];
                order[i] = order[j];
                order[j] = t;
            }
    int64_t below = d;
    for (int i : order) {
        if (size[i] <= 1) continue;
        if (stride[i] < below) return false;
        below += (size[i] - 1) * stride[i];
    }
    return true;
}

bool strides_in_range(const int64_t *stride, const int64_t *size) {
    for (int i = 0; i < 3; ++i)
        if (size[i] > 1 && stride[i] > (int64_t(1) << 42)) return false;
    return non_negative(stride);
}

bool overlap(const void *a, int64_t na, const void *b, int64_t nb, int64_t es) {
    const char *x = static_cast<const char *>(a), *y = static_cast<const char *>(b);
    return x < y + nb * es && y < x + na * es;
}

tc_status check_rotate(const tc_rotate_desc *d) {
    if (!d || !valid_dtype(d->dtype) || (d->flags & ~TC_ROTATE_BACKWARD)) return TC_ERR_INVALID_ARG;
    if (d->B < 0 || d->T < 0 || d->Hq < 1 || d->H < 0 || d->d < 1) return TC_ERR_INVALID_ARG;
    if (d->d > 128 || d->Hq > 65535 || d->H > 65535) return TC_ERR_UNSUPPORTED;
    if (d->B > (int64_t(1) << 38) || d->T > (int64_t(1) << 38)) return TC_ERR_UNSUPPORTED;
    if ((double)d->B * (double)d->T * (double)(d->Hq + d->H) * (double)d->d > 274877906944.0) return TC_ERR_UNSUPPORTED;
    const int64_t qn[3] = {d->B, d->Hq, d->T}, kn[3] = {d->B, d->H, d->T};
    if (!strides_in_range(d->q_stride, qn) || !strides_in_range(d->q_out_stride, qn) || !nested(d->q_out_stride, qn, d->d))
        return TC_ERR_INVALID_ARG;
    if (d->H && (!strides_in_range(d->k_stride, kn) || !strides_in_range(d->k_out_stride, kn) || !nested(d->k_out_stride, kn, d->d)))
        return TC_ERR_INVALID_ARG;
    return TC_OK;
}

// An output is its input (same address and strides: in place), or the two
// address ranges do not meet.
bool in_place_or_apart(const void *x, const int64_t *xs, const void *y, const int64_t *ys, const int64_t *size, int64_t d, int64_t es) {
    if (x == y) {
        for (int i = 0; i < 3; ++i)
            if (size[i] > 1 && xs[i] != ys[i]) return false;
        return true;
    }
    return !overlap(x, extent(xs, size, d), y, extent(ys, size, d), es);
}

tc_status check_cache(const tc_paged_cache *c) {
    if (!c || !valid_dtype(c->dtype)) return TC_ERR_INVALID_ARG;
    if (c->B < 1 || c->H < 1 || c->d < 1 || c->page < 1 || c->n_pages < 1 || c->max_pages < 1) return TC_ERR_INVALID_ARG;
    if (!c->k_pages || !c->v_pages || !c->table || !c->len || !c->clock) return TC_ERR_INVALID_ARG;
    if ((c->mass == nullptr) != (c->pos == nullptr)) return TC_ERR_INVALID_ARG;
    if (c->A && (!c->lambda || !c->eta)) return TC_ERR_INVALID_ARG;
    if (!aligned(c->k_pages, 16) || !aligned(c->v_pages, 16) || !aligned(c->A, 16) || !aligned(c->mass, 4) ||
        !aligned(c->pos, 4) || !aligned(c->table, 4) || !aligned(c->len, 8) || !aligned(c->clock, 8) ||
        !aligned(c->lambda, 4) || !aligned(c->eta, 4))
        return TC_ERR_INVALID_ARG;
    if (c->d > 128 || !attend_supported((int)c->d)) return TC_ERR_UNSUPPORTED;
    if (c->page % 16 || c->page > 4096 || c->B > 65535 || c->H > (int64_t(1) << 20) || c->B * c->H > (int64_t(1) << 20))
        return TC_ERR_UNSUPPORTED;
    if (c->n_pages > (int64_t(1) << 31) || c->n_pages * c->H > (int64_t(1) << 31) || c->n_pages * c->H * c->page >= (int64_t(1) << 31))
        return TC_ERR_UNSUPPORTED;
    if (c->max_pages > (int64_t(1) << 24) || c->max_pages * c->page > (int64_t(1) << 24) ||
        c->B * c->max_pages * c->page > (int64_t(1) << 36))
        return TC_ERR_UNSUPPORTED;
    return TC_OK;
}

tc_status check_heads(const tc_paged_cache *c, int64_t Hq) {
    if (Hq < 1 || Hq % c->H) return TC_ERR_INVALID_ARG;
    if (Hq / c->H > 128) return TC_ERR_UNSUPPORTED;
    return TC_OK;
}

bool cache_on_device(const tc_paged_cache *c, int dev) {
    const void *must[] = {c->k_pages, c->v_pages, c->table, c->len, c->clock};
    for (const void *p : must)
        if (!api_device_ptr(p, dev)) return false;
    const void *may[] = {c->mass, c->pos, c->A, c->A ? c->lambda : nullptr, c->A ? c->eta : nullptr};
    for (const void *p : may)
        if (p && !api_device_ptr(p, dev)) return false;
    return true;
}

CacheParams cache_params(const tc_paged_cache *c) {
    CacheParams p{};
    p.k = c->k_pages;
    p.v = c->v_pages;
    p.mass = c->mass;
    p.pos = c->pos;
    p.table = c->table;
    p.len = c->len;
    p.clock = c->clock;
    p.A = c->A;
    p.lam = c->lambda;
    p.eta = c->eta;
    p.B = (int)c->B;
    p.H = (int)c->H;
    p.page = (int)c->page;
    p.n_pages = (int)c->n_pages;
    p.max_pages = (int)c->max_pages;
    p.status = api_status_ptr();
    p.page_mul = ((uint64_t(1) << 40) + c->page - 1) / c->page;
    return p;
}

// Workspace of the attention: rows' tile prefix, partial results, scores.
struct AttendRoom {
    size_t prefix, part, z, bytes;
    AttendRoom(const tc_paged_cache *c, int64_t Hq, uint32_t flags, int sms) {
        prefix = 0;
        part = round_up((size_t)(c->B + 1) * 8);
        z = part + round_up(attend_part_bytes(c->B * c->H, (int)(Hq / c->H), (int)c->d, c->dtype, sms));
        bytes = z + ((flags & TC_CACHE_ACCUMULATE) ? round_up((size_t)(c->n_pages * c->page) * (size_t)Hq * 4) : 0);
    }
};

// Workspace of an eviction: what each row holds afterwards, sorting room.
struct EvictRoom {
    size_t row_len, sort, bytes;
    EvictRoom(const tc_paged_cache *c, int sms) {
        row_len = 0;
        sort = round_up((size_t)c->B * 8);
        bytes = sort + round_up(evict_sort_bytes(c->B * c->H, (int)c->d, c->max_pages * c->page, sms));
    }
};

// Workspace of a step: what each row holds afterwards, the rotated queries,
// their reads of A, the attention's.
struct StepRoom {
    size_t row_len, q, memo, attend, bytes;
    int slices;
    StepRoom(const tc_paged_cache *c, int64_t Hq, uint32_t flags, int sms) {
        slices = evict_slices(c->B * c->H, (int)c->d, sms);
        row_len = 0;
        q = round_up((size_t)c->B * 8);
        memo = q + round_up((size_t)(c->B * Hq * c->d) * elem(c->dtype));
        attend = memo + (c->A ? round_up((size_t)(c->B * Hq * c->d) * (size_t)slices * 4) : 0);
        bytes = attend + AttendRoom(c, Hq, flags, sms).bytes;
    }
};

tc_status check_attend(const tc_paged_cache *c, int64_t Hq, uint32_t flags) {
    tc_status st = check_cache(c);
    if (st != TC_OK) return st;
    if (flags & ~TC_CACHE_ACCUMULATE) return TC_ERR_INVALID_ARG;
    if ((flags & TC_CACHE_ACCUMULATE) && !c->mass) return TC_ERR_INVALID_ARG;
    st = check_heads(c, Hq);
    if (st != TC_OK) return st;
    const int heads = attend_heads_per_item((int)(Hq / c->H), c->dtype);
    const double items = (double)((Hq / c->H + heads - 1) / heads);
    // units of work are counted in 31 bits
    return attend_units((double)c->B * (double)c->H * items, c->max_pages * c->page) < 2147483648.0 ? TC_OK : TC_ERR_UNSUPPORTED;
}

AttendParams attend_params(const tc_paged_cache *c, int64_t Hq, const float *g, void *y, uint32_t flags, char *ws, int sms) {
    const AttendRoom room(c, Hq, flags, sms);
    AttendParams p{};
    p.c = cache_params(c);
    p.y = y;
    p.g = g;
    p.Hq = (int)Hq;
    p.G = (int)(Hq / c->H);
    p.d = (int)c->d;
    p.heads = attend_heads_per_item(p.G, c->dtype);
    p.items = (p.G + p.heads - 1) / p.heads;
    p.prefix = reinterpret_cast<int *>(ws + room.prefix);
    p.part = reinterpret_cast<float *>(ws + room.part);
    p.z = (flags & TC_CACHE_ACCUMULATE) ? reinterpret_cast<float *>(ws + room.z) : nullptr;
    p.wait_ns = api_wait_limit_ns();
    return p;
}

}  // namespace

extern "C" {

tc_status tc_rotate(const tc_rotate_desc *d, const tc_rotary *rotary, const int64_t *positions, int64_t t0,
                    const void *q, const void *k, void *q_out, void *k_out, tc_stream_t stream) {
    tc_status st = check_rotate(d);
    if (st != TC_OK) return st;
    RotateParams p{};
    if (!rotary || !make_rotary_table(rotary, d->d, &p.table)) return TC_ERR_INVALID_ARG;
    const bool empty = d->B == 0 || d->T == 0;
    const size_t es = elem(d->dtype);
    if (!empty) {
        if (!q || !q_out || (d->H && (!k || !k_out))) return TC_ERR_INVALID_ARG;
        if (!aligned(q, es) || !aligned(q_out, es) || !aligned(positions, 8)) return TC_ERR_INVALID_ARG;
        if (d->H && (!aligned(k, es) || !aligned(k_out, es))) return TC_ERR_INVALID_ARG;
        const int64_t qn[3] = {d->B, d->Hq, d->T}, kn[3] = {d->B, d->H, d->T};
        if (!in_place_or_apart(q, d->q_stride, q_out, d->q_out_stride, qn, d->d, (int64_t)es)) return TC_ERR_INVALID_ARG;
        if (d->H && !in_place_or_apart(k, d->k_stride, k_out, d->k_out_stride, kn, d->d, (int64_t)es)) return TC_ERR_INVALID_ARG;
    }
    int dev = 0, sms = 0;
    st = api_current_device(&dev, &sms);
    if (st != TC_OK) return st;
    if (empty) return TC_OK;
    const void *ptrs[] = {q, q_out, d->H ? k : nullptr, d->H ? k_out : nullptr, positions};
    for (const void *x : ptrs)
        if (x && !api_device_ptr(x, dev)) return TC_ERR_INVALID_ARG;
    p.q = q;
    p.k = k;
    p.q_out = q_out;
    p.k_out = k_out;
    p.positions = positions;
    p.t0 = t0;
    p.B = d->B;
    p.T = d->T;
    p.Hq = (int)d->Hq;
    p.H = (int)d->H;
    p.d = (int)d->d;
    for (int i = 0; i < 3; ++i) {
        p.qs[i] = d->q_stride[i];
        p.ks[i] = d->k_stride[i];
        p.qos[i] = d->q_out_stride[i];
        p.kos[i] = d->k_out_stride[i];
    }
    p.backward = (d->flags & TC_ROTATE_BACKWARD) != 0;
    return launch_rotate(p, d->dtype, sms, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? TC_OK : TC_ERR_CUDA;
}

tc_status tc_cache_append(const tc_paged_cache *c, const tc_rotary *rotary, const tc_append_args *a, tc_stream_t stream) {
    tc_status st = check_cache(c);
    if (st != TC_OK) return st;
    if (!a || a->T < 0) return TC_ERR_INVALID_ARG;
    if (a->T > (int64_t(1) << 24)) return TC_ERR_UNSUPPORTED;
    AppendParams p{};
    if (!make_rotary_table(rotary, c->d, &p.table)) return TC_ERR_INVALID_ARG;
    const size_t es = elem(c->dtype);
    if (a->q && (a->Hq < 1 || !a->q_out)) return TC_ERR_INVALID_ARG;
    if (a->q && a->Hq > 65535) return TC_ERR_UNSUPPORTED;
    if (a->mass_in && !c->mass) return TC_ERR_INVALID_ARG;
    if (a->T > 0) {
        if (!a->k || !a->v) return TC_ERR_INVALID_ARG;
        if (!aligned(a->k, es) || !aligned(a->v, es) || !aligned(a->q, es) || !aligned(a->q_out, 16) ||
            !aligned(a->counts, 8) || !aligned(a->mass_in, 4))
            return TC_ERR_INVALID_ARG;
        const int64_t kn[3] = {c->B, c->H, a->T}, qn[3] = {c->B, a->Hq, a->T};
        if (!strides_in_range(a->k_stride, kn) || !strides_in_range(a->v_stride, kn) || (a->q && !strides_in_range(a->q_stride, qn)))
            return TC_ERR_INVALID_ARG;
        if (a->q && overlap(a->q, extent(a->q_stride, qn, c->d), a->q_out, c->B * a->Hq * a->T * c->d, (int64_t)es))
            return TC_ERR_INVALID_ARG;
    }
    int dev = 0;
    st = api_current_device(&dev, nullptr);
    if (st != TC_OK) return st;
    if (!cache_on_device(c, dev)) return TC_ERR_INVALID_ARG;
    if (a->T == 0) return TC_OK;
    const void *ptrs[] = {a->k, a->v, a->q, a->q ? a->q_out : nullptr, a->counts, a->mass_in};
    for (const void *x : ptrs)
        if (x && !api_device_ptr(x, dev)) return TC_ERR_INVALID_ARG;
    p.c = cache_params(c);
    p.q = a->q;
    p.k = a->k;
    p.v = a->v;
    p.q_out = a->q_out;
    p.counts = a->counts;
    p.mass_in = a->mass_in;
    p.T = a->T;
    p.Hq = (int)a->Hq;
    p.d = (int)c->d;
    for (int i = 0; i < 3; ++i) {
        p.qs[i] = a->q_stride[i];
        p.ks[i] = a->k_stride[i];
        p.vs[i] = a->v_stride[i];
    }
    return launch_cache_append(p, c->dtype, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? TC_OK : TC_ERR_CUDA;
}

size_t tc_cache_attend_workspace_size(const tc_paged_cache *c, int64_t Hq, uint32_t flags) {
    if (check_attend(c, Hq, flags) != TC_OK) return (size_t)-1;
    return AttendRoom(c, Hq, flags, api_sm_count()).bytes;
}

tc_status tc_cache_attend(const tc_paged_cache *c, int64_t Hq, const void *q, const float *g, void *y, uint32_t flags,
                          void *workspace, size_t workspace_bytes, tc_stream_t stream) {
    tc_status st = check_attend(c, Hq, flags);
    if (st != TC_OK) return st;
    if (!q || !y || !aligned(q, 16) || !aligned(y, 16) || !aligned(g, 4) || !aligned(workspace, 16)) return TC_ERR_INVALID_ARG;
    if (g && !c->A) return TC_ERR_INVALID_ARG;
    int dev = 0, sms = 0;
    st = api_current_device(&dev, &sms);
    if (st != TC_OK) return st;
    if (!workspace || workspace_bytes < AttendRoom(c, Hq, flags, sms).bytes) return TC_ERR_WORKSPACE;
    if (!cache_on_device(c, dev)) return TC_ERR_INVALID_ARG;
    const void *ptrs[] = {q, y, workspace, g};
    for (const void *x : ptrs)
        if (x && !api_device_ptr(x, dev)) return TC_ERR_INVALID_ARG;
    AttendParams p = attend_params(c, Hq, g, y, flags, static_cast<char *>(workspace), sms);
    p.q = q;
    p.row_len = c->len;
    return launch_cache_attend(p, c->dtype, sms, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? TC_OK : TC_ERR_CUDA;
}

size_t tc_cache_evict_workspace_size(const tc_paged_cache *c) {
    if (check_cache(c) != TC_OK || !c->mass) return (size_t)-1;
    return EvictRoom(c, api_sm_count()).bytes;
}

tc_status tc_cache_evict(const tc_paged_cache *c, int64_t budget, int64_t recent, void *workspace, size_t workspace_bytes,
                         tc_stream_t stream) {
    tc_status st = check_cache(c);
    if (st != TC_OK) return st;
    if (!c->mass || budget < 1 || recent < 0 || !aligned(workspace, 16)) return TC_ERR_INVALID_ARG;
    int dev = 0, sms = 0;
    st = api_current_device(&dev, &sms);
    if (st != TC_OK) return st;
    const EvictRoom room(c, sms);
    if (!workspace || workspace_bytes < room.bytes) return TC_ERR_WORKSPACE;
    if (!cache_on_device(c, dev) || !api_device_ptr(workspace, dev)) return TC_ERR_INVALID_ARG;
    char *ws = static_cast<char *>(workspace);
    EvictParams p{};
    p.c = cache_params(c);
    p.budget = budget;
    p.recent = recent;
    p.row_len = reinterpret_cast<int64_t *>(ws + room.row_len);
    p.sort_ws = reinterpret_cast<unsigned char *>(ws + room.sort);
    p.Hq = (int)c->H;
    const cudaError_t e = launch_cache_evict(p, c->dtype, (int)c->d, sms, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? TC_OK : TC_ERR_CUDA;
}

size_t tc_cache_step_workspace_size(const tc_paged_cache *c, int64_t Hq, uint32_t flags) {
    if (check_attend(c, Hq, flags) != TC_OK || !c->mass) return (size_t)-1;
    return StepRoom(c, Hq, flags, api_sm_count()).bytes;
}

tc_status tc_cache_step(const tc_paged_cache *c, const tc_rotary *rotary, const tc_step_args *a, void *workspace,
                        size_t workspace_bytes, tc_stream_t stream) {
    if (!a) return TC_ERR_INVALID_ARG;
    tc_status st = check_attend(c, a->Hq, a->flags);
    if (st != TC_OK) return st;
    if (!c->mass || a->budget < 1 || a->recent < 0) return TC_ERR_INVALID_ARG;
    const size_t es = elem(c->dtype);
    if (!a->q || !a->k || !a->v || !a->y || !aligned(a->q, es) || !aligned(a->k, es) || !aligned(a->v, es) ||
        !aligned(a->y, 16) || !aligned(a->g, 4) || !aligned(workspace, 16))
        return TC_ERR_INVALID_ARG;
    for (int i = 0; i < 2; ++i) {
        const int64_t most = int64_t(1) << 42;
        if (a->q_stride[i] < 0 || a->k_stride[i] < 0 || a->v_stride[i] < 0 || a->q_stride[i] > most ||
            a->k_stride[i] > most || a->v_stride[i] > most)
            return TC_ERR_INVALID_ARG;
    }
    if (a->g && !c->A) return TC_ERR_INVALID_ARG;
    EvictParams e{};
    if (!make_rotary_table(rotary, c->d, &e.table)) return TC_ERR_INVALID_ARG;
    int dev = 0, sms = 0;
    st = api_current_device(&dev, &sms);
    if (st != TC_OK) return st;
    const StepRoom room(c, a->Hq, a->flags, sms);
    if (!workspace || workspace_bytes < room.bytes) return TC_ERR_WORKSPACE;
    if (!cache_on_device(c, dev)) return TC_ERR_INVALID_ARG;
    const void *ptrs[] = {a->q, a->k, a->v, a->y, workspace, a->g};
    for (const void *x : ptrs)
        if (x && !api_device_ptr(x, dev)) return TC_ERR_INVALID_ARG;
    char *ws = static_cast<char *>(workspace);
    e.c = cache_params(c);
    e.budget = a->budget;
    e.recent = a->recent;
    e.row_len = reinterpret_cast<int64_t *>(ws + room.row_len);
    e.q = a->q;
    e.k_new = a->k;
    e.v_new = a->v;
    for (int i = 0; i < 2; ++i) {
        e.qs[i] = a->q_stride[i];
        e.ks[i] = a->k_stride[i];
        e.vs[i] = a->v_stride[i];
    }
    e.q_rot = ws + room.q;
    e.memo = a->g ? reinterpret_cast<float *>(ws + room.memo) : nullptr;
    e.Hq = (int)a->Hq;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (launch_cache_step_insert(e, c->dtype, (int)c->d, room.slices, s) != cudaSuccess) return TC_ERR_CUDA;
    AttendParams p = attend_params(c, a->Hq, a->g, a->y, a->flags, ws + room.attend, sms);
    p.q = e.q_rot;
    p.row_len = e.row_len;
    p.memo = e.memo;
    p.slices = room.slices;
    p.step = true;
    return launch_cache_attend(p, c->dtype, sms, s) == cudaSuccess ? TC_OK : TC_ERR_CUDA;
}

}  // extern "C"

// C ABI of the position rotation and of the paged 8-bit caches: argument
// checks, workspace carving and the launch sequence of each call.
#include "fg_abi_paged_util.h"

static_assert(fg::kPageRows % fg::kBlockRows == 0, "pages are whole blocks");

namespace {

constexpr int kMaxAppend = 1 << 20;

// Work list of the current rows, read back (synchronous).  totals_read gets
// the first three totals when it is not null.
fg_status schedule(const fg_params* p, fg_paged_cache* c, long long* totals_read, cudaStream_t s) {
  int dev = 0, sms = 0;
  c->n_work = 0;  // no decode until the list is there
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return FG_ECUDA;
  const int Gkv = kv_count(p);
  const Sched o = sched_parts(p, c);
  const long long most = sched_max_work(Gkv, c->table_len);
  const fg::ProfileDims pd = dims(p);
  cudaError_t e = fg::launch_paged_schedule(Gkv, pd.R, c->caches, c->rows, pd.w, c->table_len,
                                            (int)most, fg::q8_slots(pd, sms), o.ranges, o.items,
                                            o.cta_first, o.totals, s);
  long long h[5] = {0, 0, 0, 0, 0};
  if (e == cudaSuccess) e = cudaMemcpyAsync(h, o.totals, sizeof(h), cudaMemcpyDeviceToHost, s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  if (e != cudaSuccess) return FG_ECUDA;
  // descriptors that overlap (never laid out by the plan) would need more items than fit
  if (h[3] < Gkv || h[3] > most || h[4] < 1 || h[4] > h[3]) return FG_EINVAL;
  c->n_work = (int32_t)h[3];
  c->n_ctas = (int32_t)h[4];
  if (totals_read)
    for (int i = 0; i < 3; ++i) totals_read[i] = h[i];
  return FG_OK;
}

}  // namespace

extern "C" {

fg_status fastgen_rope_table(const double* inv_freq, int32_t count, uint64_t* turns) {
  if (!inv_freq || !turns || count < 1) return FG_EINVAL;
  for (int32_t i = 0; i < count; ++i)
    if (!(inv_freq[i] >= 0.0) || isinf(inv_freq[i])) return FG_EINVAL;
  for (int32_t i = 0; i < count; ++i) {
    double f = inv_freq[i] / 6.283185307179586476925286766559;
    f -= floor(f);
    const double t = rint(f * 18446744073709551616.0);  // 2^64
    turns[i] = t >= 18446744073709551616.0 ? 0 : (uint64_t)t;
  }
  return FG_OK;
}

fg_status fastgen_rope(const fg_params* p, const void* Q, const void* K, const int32_t* pos,
                       const fg_rope* rope, void* Q_out, void* K_out, void* stream) {
  fg_status st = check_params(p);
  if (st != FG_OK) return st;
  fg::RopeArgs r;
  if (!rope) return FG_EINVAL;
  if ((st = check_rope(rope, p->d, &r)) != FG_OK) return st;
  if ((Q == nullptr) != (Q_out == nullptr) || (K == nullptr) != (K_out == nullptr) || (!Q && !K))
    return FG_EINVAL;
  if (!aligned(Q, 16) || !aligned(K, 16) || !aligned(Q_out, 16) || !aligned(K_out, 16) ||
      !aligned(pos, 4))
    return FG_EINVAL;
  return cuda_status(fg::launch_rope(dims(p), Q, K, pos, r, Q_out, K_out, (cudaStream_t)stream));
}

int32_t fastgen_paged_table_len(const fg_params* p, int32_t max_new_tokens) {
  if (check_params(p) != FG_OK || max_new_tokens < 0) return 0;
  const long long rows = (long long)p->n + max_new_tokens;
  if (rows > 0x7fffffffLL - fg::kPageRows) return 0;
  const long long w = ratio_count(p->r_l, p->n);
  const long long len = ((rows + fg::kPageRows - 1) / fg::kPageRows +
                         (w + fg::kPageRows - 1) / fg::kPageRows) * kv_count(p);
  return len > 0x7fffffffLL - fg::kPageRows ? 0 : (int32_t)len;
}

size_t fastgen_paged_sched_bytes(const fg_params* p, int32_t table_len) {
  if (check_params(p) != FG_OK || table_len < 1) return 0;
  const int Gkv = kv_count(p);
  const long long work = sched_max_work(Gkv, table_len);
  if (work > 0x7fffffffLL) return 0;
  return kAlign + sched_ranges_bytes(Gkv) + sched_items_bytes(work) +
         (size_t)(work + 1) * sizeof(int32_t);
}

fg_status fastgen_paged_plan(const fg_params* p, const int8_t* policy, const uint8_t* keep,
                             int32_t max_new_tokens, fg_paged_cache* cache, fg_paged_info* info,
                             void* stream) {
  fg_status st = check_params(p);
  if (st != FG_OK) return st;
  if (!policy || !keep || !info || max_new_tokens < 0) return FG_EINVAL;
  if ((st = check_layout(cache)) != FG_OK) return st;
  if (!cache->next_page || !aligned(cache->next_page, 4)) return FG_EINVAL;
  const int32_t need = fastgen_paged_table_len(p, max_new_tokens);
  if (need == 0) return FG_EINVAL;
  if (cache->table_len < need) return FG_EWORKSPACE;
  if ((st = check_sched(p, cache)) != FG_OK) return st;
  const fg::ProfileDims pd = dims(p);
  cudaStream_t s = (cudaStream_t)stream;
  const Sched o = sched_parts(p, cache);
  int2* cinfo = (int2*)o.ranges;  // the ranges' place: read before they are written
  cudaError_t e = fg::launch_group(pd, policy, keep, cinfo, s);
  if (e == cudaSuccess)
    e = fg::launch_paged_plan(pd.Gkv, pd.w, max_new_tokens, cinfo, cache->caches, cache->rows,
                              cache->page_table, cache->next_page, o.totals, s);
  if (e != cudaSuccess) return FG_ECUDA;
  long long totals[3];
  if ((st = schedule(p, cache, totals, s)) != FG_OK) return st == FG_EINVAL ? FG_ECUDA : st;
  info->pages = (int32_t)totals[0];
  info->max_pages = (int32_t)totals[1];
  info->table_used = (int32_t)totals[2];
  return FG_OK;
}

int32_t fastgen_paged_fork_table_len(const fg_params* p, int32_t max_new_tokens) {
  if (check_params(p) != FG_OK || max_new_tokens < 0 ||
      max_new_tokens > 0x7fffffff - fg::kPageRows)
    return 0;
  const long long w = ratio_count(p->r_l, p->n);
  const long long seg = (max_new_tokens + fg::kPageRows - 1) / fg::kPageRows;
  const long long len =
      ((seg > 0 ? seg : 1) + (w + fg::kPageRows - 1) / fg::kPageRows) * kv_count(p);
  return len > 0x7fffffffLL - fg::kPageRows ? 0 : (int32_t)len;
}

fg_status fastgen_paged_fork(const fg_params* p, const fg_paged_cache* prefix,
                             int32_t max_new_tokens, fg_paged_cache* cache, fg_paged_info* info,
                             void* stream) {
  fg_status st = check_params(p);
  if (st != FG_OK) return st;
  if (!prefix || !prefix->caches || !aligned(prefix->caches, 8) || !info || max_new_tokens < 0)
    return FG_EINVAL;
  if ((st = check_layout(cache)) != FG_OK) return st;
  if (!cache->next_page || !aligned(cache->next_page, 4) || cache->caches == prefix->caches)
    return FG_EINVAL;
  const int32_t need = fastgen_paged_fork_table_len(p, max_new_tokens);
  if (need == 0) return FG_EINVAL;
  if (cache->table_len < need) return FG_EWORKSPACE;
  if ((st = check_sched(p, cache)) != FG_OK) return st;
  const fg::ProfileDims pd = dims(p);
  cudaStream_t s = (cudaStream_t)stream;
  const Sched o = sched_parts(p, cache);
  int2* cinfo = (int2*)o.ranges;  // the ranges' place: read before they are written
  cudaError_t e = fg::launch_fork(pd, prefix->caches, cinfo, s);
  if (e == cudaSuccess)
    e = fg::launch_paged_plan(pd.Gkv, pd.w, max_new_tokens, cinfo, cache->caches, cache->rows,
                              cache->page_table, cache->next_page, o.totals, s);
  if (e != cudaSuccess) return FG_ECUDA;
  long long totals[3];
  if ((st = schedule(p, cache, totals, s)) != FG_OK) return st == FG_EINVAL ? FG_ECUDA : st;
  info->pages = (int32_t)totals[0];
  info->max_pages = (int32_t)totals[1];
  info->table_used = (int32_t)totals[2];
  return FG_OK;
}

fg_status fastgen_paged_schedule(const fg_params* p, fg_paged_cache* cache, void* stream) {
  fg_status st = check_params(p);
  if (st != FG_OK) return st;
  if ((st = check_layout(cache)) != FG_OK) return st;
  if ((st = check_sched(p, cache)) != FG_OK) return st;
  return schedule(p, cache, nullptr, (cudaStream_t)stream);
}

fg_status fastgen_compact_q8(const fg_params* p, const void* K, const void* V, const uint8_t* keep,
                             const fg_paged_cache* cache, int32_t* dev_err, void* stream) {
  fg_status st = check_params(p);
  if (st != FG_OK) return st;
  if ((st = check_pages(cache)) != FG_OK) return st;
  if (!K || !V || !keep || !dev_err || !aligned(K, 16) || !aligned(V, 16) || !aligned(dev_err, 4))
    return FG_EINVAL;
  return cuda_status(fg::launch_compact_q8(dims(p), K, V, keep, paged_args(p, cache, dev_err),
                                           (cudaStream_t)stream));
}

// [lists B x 2 x m][old Gkv x 2][angles B x m x d / 2]
size_t fastgen_append_q8_workspace_bytes(const fg_params* p, int32_t m) {
  if (check_params(p) != FG_OK || m < 1 || m > kMaxAppend) return 0;
  return align_up((size_t)p->B * 2 * m * sizeof(int32_t)) +
         align_up((size_t)kv_count(p) * 2 * sizeof(int32_t)) +
         align_up((size_t)p->B * m * (p->d / 2) * sizeof(float2));
}

fg_status fastgen_append_q8(const fg_params* p, const fg_paged_cache* cache, const void* k_new,
                            const void* v_new, const int32_t* new_ids, int32_t m,
                            const int32_t* n_new, const int32_t* special_ids, int32_t n_special,
                            const int32_t* punct_ids, int32_t n_punct, const int32_t* pos,
                            const fg_rope* rope, void* workspace, size_t workspace_bytes,
                            int32_t* dev_err, void* stream) {
  fg_status st = check_params(p);
  if (st != FG_OK) return st;
  if ((st = check_pages(cache)) != FG_OK) return st;
  if ((st = check_ids(special_ids, n_special)) != FG_OK) return st;
  if ((st = check_ids(punct_ids, n_punct)) != FG_OK) return st;
  if (m < 1 || m > kMaxAppend || p->B > 65535) return FG_EINVAL;
  if (!cache->next_page || !k_new || !v_new || !new_ids || !pos || !workspace || !dev_err)
    return FG_EINVAL;
  if (!aligned(cache->next_page, 4) || !aligned(cache->rows_out, 4) || !aligned(k_new, 16) ||
      !aligned(v_new, 16) || !aligned(new_ids, 4) || !aligned(n_new, 4) || !aligned(pos, 4) ||
      !aligned(workspace, kAlign) || !aligned(dev_err, 4))
    return FG_EINVAL;
  fg::AppendArgs n;
  if ((st = check_rope(rope, p->d, &n.rope)) != FG_OK) return st;
  if (workspace_bytes < fastgen_append_q8_workspace_bytes(p, m)) return FG_EWORKSPACE;
  n.k_new = k_new;
  n.v_new = v_new;
  n.ids = new_ids;
  n.n_new = n_new;
  n.pos = pos;
  n.special = special_ids;
  n.ns = n_special;
  n.punct = punct_ids;
  n.np = n_punct;
  n.m = m;
  char* ws = (char*)workspace;
  n.lists = (int32_t*)ws;
  ws += align_up((size_t)p->B * 2 * m * sizeof(int32_t));
  n.old = (int32_t*)ws;
  ws += align_up((size_t)kv_count(p) * 2 * sizeof(int32_t));
  n.angles = (float2*)ws;
  return cuda_status(fg::launch_append_q8(dims(p), paged_args(p, cache, dev_err), n,
                                          (cudaStream_t)stream));
}

// [(maximum, sum) of the scores n_work x R][outputs n_work x R x d]
size_t fastgen_decode_q8_workspace_bytes(const fg_params* p, const fg_paged_cache* cache) {
  if (check_params(p) != FG_OK || !cache || cache->n_work < 0) return 0;
  const size_t nw = (size_t)cache->n_work * group_size(p);
  return align_up(nw * 2 * sizeof(float)) + align_up(nw * p->d * sizeof(float));
}

fg_status fastgen_decode_attn_q8(const fg_params* p, const fg_paged_cache* cache, const void* q,
                                 const void* k_new, const void* v_new, const int32_t* new_ids,
                                 const int32_t* special_ids, int32_t n_special,
                                 const int32_t* punct_ids, int32_t n_punct, const int32_t* pos,
                                 const fg_rope* rope, void* out, void* workspace,
                                 size_t workspace_bytes, int32_t* dev_err, void* stream) {
  fg_status st = check_params(p);
  if (st != FG_OK) return st;
  if ((st = check_pages(cache)) != FG_OK) return st;
  if ((st = check_sched(p, cache)) != FG_OK) return st;
  if ((st = check_ids(special_ids, n_special)) != FG_OK) return st;
  if ((st = check_ids(punct_ids, n_punct)) != FG_OK) return st;
  if (!q || !pos || !out || !workspace || !dev_err || (k_new == nullptr) != (v_new == nullptr))
    return FG_EINVAL;
  if (k_new && (!new_ids || !cache->next_page || !aligned(cache->next_page, 4))) return FG_EINVAL;
  if (!aligned(cache->rows_out, 4) || !aligned(q, 16) || !aligned(k_new, 16) ||
      !aligned(v_new, 16) || !aligned(out, 16) || !aligned(new_ids, 4) || !aligned(pos, 4) ||
      !aligned(workspace, kAlign) || !aligned(dev_err, 4))
    return FG_EINVAL;
  if (!has_list(p, cache)) return FG_EINVAL;
  fg::PagedDecodeArgs n;
  if ((st = check_rope(rope, p->d, &n.rope)) != FG_OK) return st;
  if (workspace_bytes < fastgen_decode_q8_workspace_bytes(p, cache)) return FG_EWORKSPACE;
  const fg::ProfileDims pd = dims(p);
  n.q = q;
  n.k_new = k_new;
  n.v_new = v_new;
  n.ids = new_ids;
  n.pos = pos;
  n.special = special_ids;
  n.ns = n_special;
  n.punct = punct_ids;
  n.np = n_punct;
  n.out = out;
  char* ws = (char*)workspace;
  n.part_ml = (float*)ws;
  n.part_acc = (float*)(ws + align_up((size_t)cache->n_work * pd.R * 2 * sizeof(float)));
  return cuda_status(fg::launch_decode_q8(pd, paged_args(p, cache, dev_err), n,
                                          (cudaStream_t)stream));
}

}  // extern "C"

// C ABI of steps behind a shared prompt, of the rows' weights and of the cut to a
// budget: argument checks, workspace carving and launches.
#include "fg_abi_paged_util.h"

namespace {

// [own partial results: (maximum, sum), outputs][scores of the pool's rows][(maximum, sum) of the
// heads][shared caches: tile counts, queries, their factors, partial results]
struct StepParts {
  size_t ml, acc, sc, head, px[5], total;
  fg::PrefixParts prefix;
};
StepParts step_parts(const fg_params* p, const fg_paged_cache* c, bool prefix, bool scores) {
  const fg::ProfileDims pd = dims(p);
  const size_t nw = (size_t)c->n_work * pd.R;
  StepParts o;
  size_t at = 0, bytes[5] = {0, 0, 0, 0, 0};
  o.prefix = fg::PrefixParts{};
  if (prefix) o.prefix = fg::prefix_parts(pd, bytes);
  const auto put = [&](size_t size) {
    const size_t was = at;
    at += align_up(size);
    return was;
  };
  o.ml = put(nw * 2 * sizeof(float));
  o.acc = put(nw * pd.d * sizeof(float));
  o.sc = put(scores ? (size_t)c->n_pages * fg::kPageRows * pd.R * sizeof(float) : 0);
  o.head = put(scores ? (size_t)pd.G * 2 * sizeof(float) : 0);
  for (int i = 0; i < 5; ++i) o.px[i] = put(bytes[i]);
  o.total = at;
  return o;
}

// The shared caches: those of one sequence, read only, so not the ones that the step appends to.
fg_status check_prefix(const fg_paged_cache* c, const fg_paged_cache* own) {
  if (c->caches == own->caches || c->rows == own->rows || c->page_table == own->page_table)
    return FG_EINVAL;
  if (!c->page_table || !c->caches || !c->rows || c->table_len < 1) return FG_EINVAL;
  if (!c->k_pages || !c->v_pages || !c->exps || !c->pos || c->n_pages < 1) return FG_EINVAL;
  if (!aligned(c->page_table, 4) || !aligned(c->caches, 8) || !aligned(c->rows, 4) ||
      !aligned(c->k_pages, 16) || !aligned(c->v_pages, 16) || !aligned(c->exps, 8) ||
      !aligned(c->pos, 16))
    return FG_EINVAL;
  return FG_OK;
}

}  // namespace

extern "C" {

size_t fastgen_decode_q8_ex_workspace_bytes(const fg_params* p, const fg_paged_cache* cache,
                                            const fg_paged_cache* prefix, int32_t scores) {
  if (check_params(p) != FG_OK || !cache || cache->n_work < 0 || cache->n_pages < 0) return 0;
  return step_parts(p, cache, prefix != nullptr, scores != 0).total;
}

fg_status fastgen_decode_attn_q8_ex(const fg_params* p, const fg_paged_cache* cache,
                                    const fg_paged_cache* prefix, float* scores, const void* q,
                                    const void* k_new, const void* v_new, const int32_t* new_ids,
                                    const int32_t* special_ids, int32_t n_special,
                                    const int32_t* punct_ids, int32_t n_punct, const int32_t* pos,
                                    const fg_rope* rope, void* out, void* workspace,
                                    size_t workspace_bytes, int32_t* dev_err, void* stream) {
  fg_status st = check_params(p);
  if (st != FG_OK) return st;
  if ((st = check_pages(cache)) != FG_OK) return st;
  if ((st = check_sched(p, cache)) != FG_OK) return st;
  if (prefix && (st = check_prefix(prefix, cache)) != FG_OK) return st;
  if ((st = check_ids(special_ids, n_special)) != FG_OK) return st;
  if ((st = check_ids(punct_ids, n_punct)) != FG_OK) return st;
  if (!q || !pos || !out || !workspace || !dev_err || (k_new == nullptr) != (v_new == nullptr))
    return FG_EINVAL;
  if (k_new && (!new_ids || !cache->next_page || !aligned(cache->next_page, 4))) return FG_EINVAL;
  if (!aligned(cache->rows_out, 4) || !aligned(scores, 8) || !aligned(q, 16) ||
      !aligned(k_new, 16) || !aligned(v_new, 16) || !aligned(out, 16) || !aligned(new_ids, 4) ||
      !aligned(pos, 4) || !aligned(workspace, kAlign) || !aligned(dev_err, 4))
    return FG_EINVAL;
  if (!has_list(p, cache)) return FG_EINVAL;
  fg::StepArgs n;
  if ((st = check_rope(rope, p->d, &n.rope)) != FG_OK) return st;
  const fg::ProfileDims pd = dims(p);
  const StepParts o = step_parts(p, cache, prefix != nullptr, scores != nullptr);
  if (workspace_bytes < o.total) return FG_EWORKSPACE;
  char* ws = (char*)workspace;
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
  n.part_ml = (float*)(ws + o.ml);
  n.part_acc = (float*)(ws + o.acc);
  n.row_w = scores;
  n.row_sc = scores ? (float*)(ws + o.sc) : nullptr;
  n.head_ml = scores ? (float*)(ws + o.head) : nullptr;
  n.beside = prefix ? 1 : 0;
  fg::PrefixParts px = o.prefix;
  fg::PagedArgs pre = {};
  if (prefix) {
    px.cum = (long long*)(ws + o.px[0]);
    px.q = (uint8_t*)(ws + o.px[1]);
    px.qf = (float*)(ws + o.px[2]);
    px.ml = (float*)(ws + o.px[3]);
    px.acc = (float*)(ws + o.px[4]);
    fg_paged_cache c = *prefix;
    c.sched = nullptr;
    pre = paged_args(p, &c, dev_err);
  }
  return cuda_status(
      fg::launch_step_q8(pd, paged_args(p, cache, dev_err), n, pre, px, (cudaStream_t)stream));
}

fg_status fastgen_paged_clear(const fg_params* p, const fg_paged_cache* cache, int32_t* dev_err,
                              void* stream) {
  fg_status st = check_params(p);
  if (st != FG_OK) return st;
  if ((st = check_pages(cache)) != FG_OK) return st;
  if (!aligned(cache->rows_out, 4) || !dev_err || !aligned(dev_err, 4)) return FG_EINVAL;
  return cuda_status(fg::launch_paged_clear(dims(p), paged_args(p, cache, dev_err), cache->rows,
                                            (cudaStream_t)stream));
}

fg_status fastgen_scores_q8(const fg_params* p, const fg_paged_cache* cache, float* scores,
                            const float* colsum, const int32_t* ids, int32_t m,
                            const int32_t* n_new, const int32_t* pos, const int32_t* special_ids,
                            int32_t n_special, int32_t* dev_err, void* stream) {
  fg_status st = check_params(p);
  if (st != FG_OK) return st;
  if ((st = check_pages(cache)) != FG_OK) return st;
  if ((st = check_ids(special_ids, n_special)) != FG_OK) return st;
  if (!scores || !ids || m < 1 || !dev_err) return FG_EINVAL;
  if (!aligned(scores, 4) || !aligned(colsum, 4) || !aligned(ids, 4) || !aligned(n_new, 4) ||
      !aligned(pos, 4) || !aligned(dev_err, 4))
    return FG_EINVAL;
  fg::ScoreArgs n;
  n.scores = scores;
  n.colsum = colsum;
  n.ids = ids;
  n.n_new = n_new;
  n.pos = pos;
  n.special = special_ids;
  n.ns = n_special;
  n.m = m;
  return cuda_status(fg::launch_scores_q8(dims(p), paged_args(p, cache, dev_err), n,
                                          (cudaStream_t)stream));
}

// [rows that move Gkv][the row that comes to each place, and lists of them: 2 x Gkv x budget]
size_t fastgen_evict_q8_workspace_bytes(const fg_params* p, int32_t budget) {
  if (check_params(p) != FG_OK || budget < 1 || budget % fg::kBlockRows != 0) return 0;
  return align_up((size_t)kv_count(p) * sizeof(int32_t)) +
         align_up((size_t)kv_count(p) * budget * 2 * sizeof(int32_t));
}

fg_status fastgen_evict_q8(const fg_params* p, const fg_paged_cache* cache, float* scores,
                           int32_t budget, int32_t recent, const int32_t* pos, void* workspace,
                           size_t workspace_bytes, int32_t* dev_err, void* stream) {
  fg_status st = check_params(p);
  if (st != FG_OK) return st;
  if ((st = check_pages(cache)) != FG_OK) return st;
  if (budget < 1 || budget % fg::kBlockRows != 0 || recent < 0 || recent > budget)
    return FG_EINVAL;
  if (!scores || !pos || !workspace || !dev_err) return FG_EINVAL;
  if (!aligned(cache->rows_out, 4) || !aligned(scores, 4) || !aligned(pos, 4) ||
      !aligned(workspace, kAlign) || !aligned(dev_err, 4))
    return FG_EINVAL;
  if (workspace_bytes < fastgen_evict_q8_workspace_bytes(p, budget)) return FG_EWORKSPACE;
  fg::EvictArgs n;
  n.scores = scores;
  n.pos = pos;
  n.budget = budget;
  n.recent = recent;
  n.caches = kv_count(p);
  n.moves = (int32_t*)workspace;
  n.src = (int32_t*)((char*)workspace + align_up((size_t)kv_count(p) * sizeof(int32_t)));
  return cuda_status(fg::launch_evict_q8(dims(p), paged_args(p, cache, dev_err), n,
                                         (cudaStream_t)stream));
}

}  // extern "C"

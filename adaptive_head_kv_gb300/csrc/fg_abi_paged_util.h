// Argument checks and the work list's layout shared by the C-ABI files of the
// paged 8-bit caches.
#pragma once

#include "fg_abi_util.h"
#include "fg_paged.cuh"

namespace {

// rope may be null (no rotation).
fg_status check_rope(const fg_rope* r, int d, fg::RopeArgs* out) {
  out->turns = nullptr;
  out->rot = 0;
  out->style = FG_ROPE_INTERLEAVED;
  if (!r) return FG_OK;
  if (!r->turns || !aligned(r->turns, 8)) return FG_EINVAL;
  if (r->rot_dim < 16 || r->rot_dim > d || r->rot_dim % 16 != 0) return FG_EINVAL;
  if (r->style != FG_ROPE_INTERLEAVED && r->style != FG_ROPE_HALF) return FG_EINVAL;
  out->turns = (const unsigned long long*)r->turns;
  out->rot = r->rot_dim;
  out->style = r->style;
  return FG_OK;
}

// sched: [totals: 256 bytes][ranges int4 x Gkv][items][first items of the thread blocks]
size_t sched_ranges_bytes(int Gkv) { return align_up((size_t)Gkv * sizeof(int4)); }
size_t sched_items_bytes(long long work) { return align_up((size_t)work * sizeof(fg::PagedItem)); }

// Work items a table of table_len entries can need: items of kItemPages
// pages, one that a cache leaves over, one that the cut of a length adds.
long long sched_max_work(int Gkv, int32_t table_len) {
  return (long long)table_len / fg::kItemPages + 2LL * Gkv + 1;
}

struct Sched {
  long long* totals;
  int4* ranges;
  fg::PagedItem* items;
  int32_t* cta_first;
};
Sched sched_parts(const fg_params* p, const fg_paged_cache* c) {
  char* s = (char*)c->sched;
  Sched o;
  o.totals = (long long*)s;
  o.ranges = (int4*)(s + kAlign);
  s += kAlign + sched_ranges_bytes(kv_count(p));
  o.items = (fg::PagedItem*)s;
  o.cta_first = (int32_t*)(s + sched_items_bytes(sched_max_work(kv_count(p), c->table_len)));
  return o;
}

fg_status check_sched(const fg_params* p, const fg_paged_cache* c) {
  if (!c->sched || !aligned(c->sched, kAlign)) return FG_EINVAL;
  const size_t need = fastgen_paged_sched_bytes(p, c->table_len);
  if (need == 0) return FG_EINVAL;
  if (c->sched_bytes < 0 || (size_t)c->sched_bytes < need) return FG_EWORKSPACE;
  return FG_OK;
}

// What every call needs of the table and the descriptors.
fg_status check_layout(const fg_paged_cache* c) {
  if (!c || !c->page_table || !c->caches || !c->rows || c->table_len < 1) return FG_EINVAL;
  if (!aligned(c->page_table, 4) || !aligned(c->caches, 8) || !aligned(c->rows, 4))
    return FG_EINVAL;
  return FG_OK;
}

fg_status check_pages(const fg_paged_cache* c) {
  fg_status st = check_layout(c);
  if (st != FG_OK) return st;
  if (!c->k_pages || !c->v_pages || !c->exps || !c->pos || c->n_pages < 1) return FG_EINVAL;
  if (!aligned(c->k_pages, 16) || !aligned(c->v_pages, 16) || !aligned(c->exps, 8) ||
      !aligned(c->pos, 16))
    return FG_EINVAL;
  return FG_OK;
}

fg::PagedArgs paged_args(const fg_params* p, const fg_paged_cache* c, int32_t* dev_err) {
  fg::PagedArgs a;
  a.kp = (uint8_t*)c->k_pages;
  a.vp = (uint8_t*)c->v_pages;
  a.exps = c->exps;
  a.pos = c->pos;
  a.table = c->page_table;
  a.caches = c->caches;
  a.rows = c->rows;
  a.rows_out = c->rows_out ? c->rows_out : c->rows;
  a.next_page = c->next_page;
  if (c->sched) {
    const Sched o = sched_parts(p, c);
    a.ranges = o.ranges;
    a.items = o.items;
    a.cta_first = o.cta_first;
    a.totals = o.totals;
  } else {
    a.ranges = nullptr;
    a.items = nullptr;
    a.cta_first = nullptr;
    a.totals = nullptr;
  }
  a.n_pages = c->n_pages;
  a.table_len = c->table_len;
  a.n_work = c->n_work;
  a.n_ctas = c->n_ctas;
  a.max_w = ratio_count(p->r_l, p->n);
  a.dev_err = dev_err;
  return a;
}

// A work list is there: one item a cache at least, no thread block without one.
inline bool has_list(const fg_params* p, const fg_paged_cache* c) {
  return c->n_work >= kv_count(p) && c->n_work <= sched_max_work(kv_count(p), c->table_len) &&
         c->n_ctas >= 1 && c->n_ctas <= c->n_work;
}

}  // namespace

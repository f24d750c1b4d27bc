// Host checks and work partition shared by the attention step's kernels.
#pragma once

#include "lk_attn.h"
#include "lk_device.cuh"
#include "lk_host.h"

namespace lkattn {

inline int log2_of(int p) {
  int n = 0;
  while ((1 << n) < p) ++n;
  return n;
}

inline lk_status check_cache(const lk_kv_cache* c, int n_q) {
  if (!c) return LK_ERR_ARG;
  if (c->type < LK_KV_F16 || c->type > LK_KV_Q8) return LK_ERR_ARG;
  if (c->head_dim != 64 && c->head_dim != 128) return LK_ERR_SHAPE;
  if (c->page < 16 || c->page > 1024 || (c->page & (c->page - 1))) return LK_ERR_SHAPE;
  if (c->n_kv < 1 || c->n_pages < 1 || n_q < c->n_kv || n_q % c->n_kv || n_q > 4096) return LK_ERR_SHAPE;
  if (!c->k || !c->v || (c->type == LK_KV_Q8 && (!c->ks || !c->vs))) return LK_ERR_ARG;
  if (!lkh::aligned(c->k, 16) || !lkh::aligned(c->v, 16)) return LK_ERR_ALIGN;
  if (c->type == LK_KV_Q8 && (!lkh::aligned(c->ks, 16) || !lkh::aligned(c->vs, 16))) return LK_ERR_ALIGN;
  return LK_OK;
}

// B, R, table and lens (the pointers only where there are rows)
inline lk_status check_rows(const lk_kv_cache* c, const int32_t* table, int table_w, const int32_t* lens, int B,
                            int R) {
  if (B < 0 || R < 0 || B > LK_MAX_BATCH || R > LK_MAX_BATCH || B * R > LK_MAX_BATCH) return LK_ERR_SHAPE;
  if (table_w < 0 || (long)table_w * c->page > 0x40000000L) return LK_ERR_SHAPE;
  if (B == 0 || R == 0) return LK_OK;
  if (!lens || (table_w > 0 && !table)) return LK_ERR_ARG;
  if (!lkh::aligned(lens, 4) || (table && !lkh::aligned(table, 4))) return LK_ERR_ALIGN;
  return LK_OK;
}

}  // namespace lkattn

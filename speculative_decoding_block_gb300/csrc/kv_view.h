// kv_view.h -- what the single-token serving operators (decode attention,
// eviction) need of a cache object: its shape, its device memory and the
// tensor maps of its pools.
#pragma once

#include "vsd_common.cuh"

namespace vsd {

struct KvView {
  const vsd_model* model;
  int layers, n_q, n_kv, hd;
  int max_batch, max_tokens, num_pages, ppr, sms;
  __nv_bfloat16 *k_pool, *v_pool;  // [layers][num_pages][n_kv][16][hd]
  const int* page_table;           // [max_batch][ppr]
  int* status;
  CUtensorMap tm_k, tm_v;  // rows of the pools, boxes of 16 rows x 64 columns, 128-byte swizzle
};
KvView kv_view(const vsd_kv* kv);

}  // namespace vsd

// What stands behind the library's handles, for the files that hold their entry points.
#pragma once

#include <cuda.h>

#include "gdn_internal.h"

struct gdn_pool {
  gdn::PoolView view;
  gdn_pool_desc desc;
  int device;
  int sm_count;
  bool has_tmap;
  alignas(64) CUtensorMap tmap;  // the state as a [rows][dk] float32 tensor (TMA)
  cudaMemPool_t work_pool;       // stream-ordered prefill workspaces (kept until destroy)
};

struct gdn_kv {
  gdn::KVView view;
  gdn_kv_desc desc;
  int device;
  int sm_count;
  alignas(64) CUtensorMap k_map, v_map;  // see gdn::KVHost
  gdn::KVWork work;
};

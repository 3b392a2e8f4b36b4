// attn_tree_tc_host.cpp — the kernel for many rows.
#include "attn_host.h"

#include "kda_attn_tree_tc.cu"

static const bool ready = (emu::shared_memory = kda::smem_raw, true);

// Device-side status bits shared by the kernels and the host library.  The
// kernels OR these into a 32-bit word in the caller's workspace; the host maps
// the word to a coda_status with coda_get_status().
#pragma once

#define CODA_DEV_TIMEOUT 0x1         // a bounded mbarrier wait ran out
#define CODA_DEV_LABEL_RANGE 0x2     // a label outside [0, V) that is not ignore_index
#define CODA_DEV_POSITION_RANGE 0x4  // a RoPE position outside [0, max_pos)
#define CODA_DEV_SEQLEN_RANGE 0x8    // sequence offsets that fall or leave the tensor, or a length beyond its page table
#define CODA_DEV_PAGE_RANGE 0x10     // a cache slot or page index outside the cache
#define CODA_DEV_TREE_RANGE 0x20     // a tree's parent, path or size that names no tree
#define CODA_DEV_PROB_RANGE 0x40     // probabilities of a row that sum to 16 or more

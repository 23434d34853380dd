// The notes that the tree attention leaves for its merge, and what the merge takes from them.  Plain
// C++, for the kernels and for host programs.
#pragma once

#ifdef __CUDACC__
#define MSA_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define MSA_HOST_DEVICE inline
#endif

namespace msa {

// One cut item (a query's block of drafts under one KV head): the groups first .. last of n_kv CTAs
// share its tiles.  The parts of the groups behind the first lie in slot 2 (group n_kv + head), the
// first group's in slot `slot`.
struct MergeNote {
  int query;  // -1: nothing to merge
  int draft, head, n_draft;
  int first, last, slot;
};

// Is the note one that the attention kernel writes for a call of these sizes?  Notes stand in the
// caller's workspace and are written in the course of the work: a CTA that gave up waiting leaves
// the ones of its later items as the workspace had them.  Whatever stands there, the merge of a note
// that passes reads parts and writes output rows inside their buffers and ends: query, draft and head
// index the output, groups and slot the parts.
MSA_HOST_DEVICE bool merge_note_ok(const MergeNote& n, int B, int M, int n_kv, int groups) {
  return n.query >= 0 && n.query < B && n.draft >= 0 && n.draft < M && n.head >= 0 && n.head < n_kv && n.first >= 0 &&
         n.first < n.last && n.last < groups && n.slot >> 1 == n.first * n_kv + n.head;
}

}  // namespace msa

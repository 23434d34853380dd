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
  // (unsigned: a negative number is out of range too; one predicate, no chain of branches)
  const auto below = [](int v, int end) { return static_cast<unsigned>(v) < static_cast<unsigned>(end); };
  return below(n.query, B) & below(n.draft, M) & below(n.head, n_kv) & below(n.first, n.last) & below(n.last, groups) &
         (n.slot >> 1 == n.first * n_kv + n.head);
}

}  // namespace msa

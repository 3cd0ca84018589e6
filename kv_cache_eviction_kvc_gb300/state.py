"""Device-memory plumbing for a decode stream: allocates the cache, moment,
workspace and output tensors with torch and calls the libkvc entry points
through the binding.  No arithmetic of the method happens here."""
from __future__ import annotations

import torch

from . import kvc as K_


class DecodeState:
    """Cache + moments + workspace of U units on one device."""

    def __init__(self, U: int, G: int, cap: int, L: int, *, rule: int = K_.RULE_EMA,
                 alpha: float = 0.9, refresh_period: int = 1,
                 correction: int = K_.CORR_FIRST_ORDER, votes: bool = False,
                 kmax: int = 1, device="cuda", d: int = 128, merge_recent: int | None = None,
                 budgets: bool = False, chain=None):
        self.U, self.G, self.cap, self.L, self.d = U, G, cap, L, d
        self.device = torch.device(device)
        # per-unit budgets (a cache handed over from a prefill selection);
        # the tensor lives as long as the parameters that point at it
        self.budget = (torch.full((U,), L, dtype=torch.int32, device=self.device)
                       if budgets else None)
        self.params = K_.make_params(U, G, cap, L, rule, alpha, refresh_period, correction, d,
                                     merge_recent, self.budget, chain)
        self.merge = merge_recent is not None
        if self.merge and not votes:
            raise ValueError("ZIP-merging needs per-slot votes (votes=True)")
        dev = self.device
        self.K = torch.zeros(U, cap, d, dtype=torch.bfloat16, device=dev)
        self.V = torch.zeros(U, cap, d, dtype=torch.bfloat16, device=dev)
        self.votes = torch.ones(U, cap, dtype=torch.int32, device=dev) if votes else None
        self.pos = torch.full((U, cap), -1, dtype=torch.int32, device=dev)
        self.util = torch.full((U, cap), float("inf"), dtype=torch.float64, device=dev)
        self.len = torch.zeros(U, dtype=torch.int32, device=dev)
        self.n = torch.zeros(U, dtype=torch.float32, device=dev)
        self.mu_k = torch.zeros(U, d, dtype=torch.float32, device=dev)
        self.mu_v = torch.zeros(U, d, dtype=torch.float32, device=dev)
        self.C = torch.zeros(U, d, d, dtype=torch.float32, device=dev)
        nbytes = K_.kvc_decode_workspace_size(self.params)
        if nbytes == 0:
            raise K_.KvcError(1, "invalid decode parameters")
        self.ws = torch.empty(nbytes, dtype=torch.uint8, device=dev)
        K_.kvc_decode_workspace_init(self.params, self.ws)
        self.o = torch.zeros(U, G, d, dtype=torch.float32, device=dev)
        self.probs = torch.zeros(U, cap, dtype=torch.float64, device=dev)
        self.lse = torch.zeros(U, G, dtype=torch.float32, device=dev)
        self.f_all = torch.zeros(U, G, d, dtype=torch.float32, device=dev)
        self.f_R = torch.zeros(U, G, d, dtype=torch.float32, device=dev)
        self.logZ_R = torch.zeros(U, G, dtype=torch.float32, device=dev)
        self.n_evict = torch.zeros(U, dtype=torch.int32, device=dev)
        self.partner_pos = torch.full((U,), -1, dtype=torch.int32, device=dev)
        self.scores = (torch.zeros(U, cap, dtype=torch.float64, device=dev)
                       if rule == K_.RULE_MI else None)
        self.set_kmax(kmax)

    # --------------------------------------------------------------- helpers
    def set_kmax(self, kmax: int):
        kmax = max(1, int(kmax))
        if getattr(self, "kmax", 0) != kmax:
            self.kmax = kmax
            self.evict_idx = torch.full((self.U, kmax), -1, dtype=torch.int32, device=self.device)
            self.evict_pos = torch.full((self.U, kmax), -1, dtype=torch.int32, device=self.device)

    @property
    def cache(self) -> K_.kvc_cache:
        return K_.make_cache(self.K, self.V, self.votes, self.pos, self.util, self.len)

    @property
    def moments(self) -> K_.kvc_moments:
        return K_.make_moments(self.n, self.mu_k, self.mu_v, self.C)

    def load_prefill(self, K, V, votes, pos, length):
        """Copy a prefill cache laid out [U][>=N][d] into the state."""
        n = K.shape[1]
        if K.data_ptr() != self.K.data_ptr():      # drawn in place: nothing to copy
            self.K[:, :n].copy_(K)
        if V.data_ptr() != self.V.data_ptr():
            self.V[:, :n].copy_(V)
        if self.votes is not None and votes is not None:
            self.votes[:, :n].copy_(votes[:, :n])
        self.pos[:, :n].copy_(pos[:, :n])
        self.util.fill_(float("inf"))
        self.len.copy_(length)
        for t in (self.n, self.mu_k, self.mu_v, self.C):
            t.zero_()

    def load_handoff(self, N, keep, K_src, V_src, votes_src=None, util_init=None):
        """Start the stream from a prefill selection (kvc_prefill_handoff):
        keep [U][N] uint8, K_src / V_src [U][N][d]; the per-unit budgets land
        in self.budget.  Returns the device status of the call."""
        ws = torch.empty(K_.kvc_prefill_handoff_workspace_size(self.U, N), dtype=torch.uint8,
                         device=self.device)
        K_.kvc_prefill_handoff(self.params, N, keep, K_src, V_src, votes_src, util_init,
                               self.cache, self.moments, self.budget, ws)
        return K_.kvc_get_device_status(ws)

    def device_status(self) -> int:
        return K_.kvc_get_device_status(self.ws)

    # --------------------------------------------------------------- steps
    def step(self, t: int, new_pos: int, q, k_new, v_new, max_len: int, emit_probs=True,
             stream=None, o=None):
        """Fused kvc_decode_step (falls back to the five-call sequence inside
        the library when the step is not in the steady state).  `o` may name
        another [U][G][d] fp32 output buffer."""
        self.set_kmax(max_len - self.L)
        K_.kvc_decode_step(self.params, t, new_pos, max_len, q, k_new, v_new, self.cache,
                           self.moments, self.o if o is None else o,
                           self.probs if emit_probs else None,
                           self.kmax, self.evict_idx, self.evict_pos, self.n_evict, self.ws,
                           stream)

    def step_calls(self, t: int, new_pos: int, q, k_new, v_new, max_len: int, stream=None):
        """The five entry points in order (attend, aggregate_evict,
        moment_update, correct, compact), with zip_merge after aggregate_evict
        in merge mode and mi_scores before it under the moment-informed rule
        (mi_evict in place of scores, aggregate and fold when that rule
        removes several slots)."""
        self.set_kmax(max_len - self.L)
        c = self.cache
        K_.kvc_decode_attend(self.params, t, new_pos, max_len, q, k_new, v_new, c, self.lse,
                             self.f_all, self.probs, self.ws, stream)
        mi = self.params.rule == K_.RULE_MI          # the rule of this step
        if mi and max_len - self.L > 1:
            # MomentKV Algorithm 1's loop: score, evict the lowest, fold, again
            K_.kvc_mi_evict(self.params, max_len, c, self.moments, self.lse, self.kmax,
                            self.evict_idx, self.evict_pos, self.n_evict, self.ws, stream)
            K_.kvc_correct(self.params, q, c, self.kmax, self.evict_idx, self.n_evict, self.lse,
                           self.f_all, self.moments, self.o, self.f_R, self.logZ_R, self.ws,
                           stream)
            K_.kvc_compact(self.params, c, self.kmax, self.evict_idx, self.n_evict, self.ws,
                           stream)
            return
        agg_in = self.probs
        if mi:
            K_.kvc_mi_scores(self.params, c, self.moments, max_len, self.probs, self.scores, stream)
            agg_in = self.scores
        K_.kvc_aggregate_evict(self.params, t, agg_in, c, self.kmax, self.evict_idx,
                               self.evict_pos, self.n_evict, self.ws, stream)
        if self.merge:
            K_.kvc_zip_merge(self.params, new_pos, q, c, self.kmax, self.evict_idx, self.n_evict,
                             self.partner_pos, self.ws, stream)
        K_.kvc_moment_update(self.params, c, self.kmax, self.evict_idx, self.n_evict,
                             self.moments, self.ws, stream)
        K_.kvc_correct(self.params, q, c, self.kmax, self.evict_idx, self.n_evict, self.lse,
                       self.f_all, self.moments, self.o, self.f_R, self.logZ_R, self.ws, stream)
        K_.kvc_compact(self.params, c, self.kmax, self.evict_idx, self.n_evict, self.ws, stream)

    # --------------------------------------------------------------- drafted tokens
    def verify(self, tree: K_.kvc_tree, q, k_tree, v_tree, max_len: int, stream=None):
        """Attention of a tree of drafted tokens over the cache (the cache
        does not change): q [U][T][G][d], k_tree / v_tree [U][T][d].  Returns
        (o [U][T][G][d] bf16, lse [U][T][G] fp32), buffers of the state that
        the next call with the same T writes again.  The first call with a T
        allocates (make it before capturing one into a graph) what the state
        then keeps: o and lse, and a workspace of 520 bytes for each of
        (U ceil(T G / 256) + 152) min(T G, 256) rows (1024 units, G = 4,
        T = 16: 17 and 39 MB).  A loop over many T keeps buffers of each."""
        b = self._tree_buffers(tree.T, True, stream)
        K_.kvc_tree_attend(self.params, max_len, tree, q, k_tree, v_tree, self.cache, self.moments,
                           b["o"], b["lse"], b["ws"], stream)
        return b["o"], b["lse"]

    def accept(self, tree: K_.kvc_tree, path: K_.kvc_path, q, k_tree, v_tree, max_len: int,
               row_weight=None, refresh=True, stream=None):
        """After verify of the same tree: the accepted path joins the cache.
        With refresh the utilities take the weight the accepted tokens gave
        (row_weight: fp32 [trees][A] or None; held in fp64, as a step's
        probabilities are); the lowest go until every unit is at its budget.
        self.n_evict has the counts, self.tree_evict the slots and positions
        ([2][U][most victims of this call]); tree_status() has the errors of
        both calls."""
        b = self._tree_buffers(tree.T, False)
        S = None
        if refresh:
            S = self.tree_S
            K_.kvc_tree_weights(self.params, max_len, tree, path, row_weight, q, k_tree,
                                b["lse"], self.cache, S, b["ws"], stream)
        # as many victims as there can be: fewer leave room for more units at once
        kmax = K_.TREE_MAX
        if self.budget is None:
            kmax = min(kmax, max(1, max_len + path.A - self.L))
        self.tree_evict = self._tree_evict[:2 * self.U * kmax].view(2, self.U, kmax)
        K_.kvc_tree_commit(self.params, max_len, tree, path, k_tree, v_tree, S, self.cache,
                           self.moments, kmax, self.tree_evict[0], self.tree_evict[1],
                           self.n_evict, self.ws, stream)

    def _tree_buffers(self, T, make, stream=None):
        """What verify and accept of trees of T tokens use; kept for each T
        (a captured graph goes on using them)."""
        trees = self.__dict__.setdefault("_trees", {})
        if T not in trees:
            if not make:
                raise ValueError(f"no tree of T = {T} tokens has been verified")
            nbytes = K_.kvc_tree_workspace_size(self.params, T)
            if nbytes == 0:
                raise ValueError(f"no trees of T = {T} tokens")
            dev = self.device
            if not trees:
                # fp64, as the utilities: over sharp attention most weights are below
                # fp32's range, and the victims go by their order
                self.tree_S = torch.zeros(self.U, self.cap, dtype=torch.float64, device=dev)
                self._tree_evict = torch.full((2 * self.U * K_.TREE_MAX,), -1, dtype=torch.int32,
                                              device=dev)
            trees[T] = dict(
                ws=torch.zeros(nbytes, dtype=torch.uint8, device=dev),
                o=torch.zeros(self.U, T, self.G, self.d, dtype=torch.bfloat16, device=dev),
                lse=torch.zeros(self.U, T, self.G, dtype=torch.float32, device=dev))
            if stream is not None:
                # the fills above are on the current stream: the call's waits for them
                if not hasattr(stream, "wait_stream"):       # a handle; 0: the default stream
                    handle = int(getattr(stream, "cuda_stream", stream))
                    stream = (torch.cuda.ExternalStream(handle, dev) if handle
                              else torch.cuda.default_stream(dev))
                stream.wait_stream(torch.cuda.current_stream(dev))
        return trees[T]

    def tree_status(self) -> int:
        """The first error that a verify or accept recorded and that has not
        been read yet (0: none).  accept's commit records in the decode
        stream's workspace, as the steps do: an error there is returned here
        or by device_status(), whichever is asked first."""
        trees = self.__dict__.get("_trees", {})
        for ws in [b["ws"] for b in trees.values()] + ([self.ws] if trees else []):
            status = K_.kvc_get_device_status(ws)
            if status:
                return status
        return 0


class PagedState:
    """A cache in pages of `seqs` sequences of `heads` units (heads = 1: a table
    and a length per unit), with the pool's bookkeeping: pages are taken from a
    free list on the host as sequences grow and go back when they end.  It is
    one layer's; the calls themselves leave the lengths alone, so that layers may
    share a table and a length (kvc.make_pages).  Lengths advance by the rows that
    were taken: a sequence that a call refuses (status()) keeps its length.  A
    place that holds no pages is free: steps leave it out.  Calls run on the
    current stream."""

    def __init__(self, seqs: int, heads: int, G: int, max_len: int, *, page: int = 64,
                 e4m3: bool = True, n_pages: int | None = None, device="cuda", d: int = 128):
        self.seqs, self.heads, self.G, self.page, self.d = seqs, heads, G, page, d
        self.device = dev = torch.device(device)
        stride = -(-max_len // page)
        n_pages = seqs * stride if n_pages is None else n_pages
        shape = (n_pages, heads, page, d)
        dtype = torch.float8_e4m3fn if e4m3 else torch.bfloat16
        self.K = torch.zeros(shape, dtype=dtype, device=dev)
        self.V = torch.zeros(shape, dtype=dtype, device=dev)
        self.k_scale = torch.zeros(shape[:3], device=dev) if e4m3 else None
        self.v_scale = torch.zeros(shape[:3], device=dev) if e4m3 else None
        self.table = torch.full((seqs, stride), -1, dtype=torch.int32, device=dev)
        self.len = torch.zeros(seqs, dtype=torch.int32, device=dev)
        self.room = torch.zeros(seqs, dtype=torch.int32, device=dev)    # slots of the pages held
        self.pages = K_.make_pages(self.K, self.V, self.k_scale, self.v_scale, self.table, self.len)
        nbytes = K_.kvc_page_workspace_size(self.pages, G)
        if nbytes == 0:
            raise K_.KvcError(1, K_.kvc_last_error() or "invalid page parameters")
        self.ws = torch.zeros(nbytes, dtype=torch.uint8, device=dev)
        self.o = torch.zeros(seqs * heads, G, d, dtype=torch.bfloat16, device=dev)
        self.lse = torch.zeros(seqs * heads, G, dtype=torch.float32, device=dev)
        self._free = list(range(n_pages - 1, -1, -1))
        self._held = [[] for _ in range(seqs)]

    # --------------------------------------------------------------- pages
    def reserve(self, lengths):
        """Pages for lengths[s] slots of every sequence (a host list; what a
        sequence has already stays).  A pool without enough raises and nothing
        changes."""
        if len(lengths) != self.seqs:
            raise ValueError(f"{len(lengths)} lengths for {self.seqs} sequences")
        want = [max(0, -(-int(n) // self.page) - len(h)) for n, h in zip(lengths, self._held)]
        for n, h, w in zip(lengths, self._held, want):
            if len(h) + w > self.table.shape[1]:
                raise ValueError(f"{n} slots are more than a table of {self.table.shape[1]} pages holds")
        if sum(want) > len(self._free):
            raise RuntimeError(f"the pool has {len(self._free)} free pages, {sum(want)} are needed")
        at, value = [], []
        for s, w in enumerate(want):
            for _ in range(w):
                at.append(s * self.table.shape[1] + len(self._held[s]))
                self._held[s].append(self._free.pop())
                value.append(self._held[s][-1])
        if at:
            i = torch.tensor([at, value], dtype=torch.int64).to(self.device)
            self.table.view(-1).index_copy_(0, i[0], i[1].to(torch.int32))
            self.room.copy_(torch.tensor([len(h) * self.page for h in self._held], dtype=torch.int32))

    def release(self, s: int):
        """The pages of sequence s go back to the pool; its length becomes 0, its
        place free."""
        self._free += reversed(self._held[s])
        self._held[s] = []
        self.table[s].fill_(-1)
        self.len[s].zero_()
        self.room[s].zero_()

    # --------------------------------------------------------------- calls
    def write(self, k, v, count=None):
        """Rows k, v [U][T][d] behind what the sequences hold (count: int32
        [seqs], None: T rows each); the lengths advance.  Reserve their pages
        before: a sequence without room for its rows keeps its length."""
        K_.kvc_page_write(self.pages, self.len, count, k, v, self.ws)
        T = k.shape[1]
        if count is None:
            self.len.add_((self.len <= self.room - T) * T)
        else:
            taken = (count >= 0) & (count <= T) & (self.len + count <= self.room)
            self.len.add_(torch.where(taken, count, 0))

    def step(self, q, k_new, v_new, max_len: int):
        """One token per sequence that holds pages: k_new, v_new [U][d] join the
        cache, q [U][G][d] attends over it; the lengths advance.  max_len bounds
        the new lengths; a sequence that has no slot left, or would pass max_len,
        keeps its length.  Returns (o [U][G][d] bf16, lse [U][G] fp32), written
        again by the next call (of free places and refused sequences: as they
        were)."""
        K_.kvc_page_attend(self.pages, max_len, q, k_new, v_new, self.o, self.lse, self.ws)
        self.len.add_(self.len < self.room.clamp(max=int(max_len)))
        return self.o, self.lse

    def read(self, M: int, slots=None, count=None):
        """bf16 rows (k, v [U][M][d]) of slots [U][M] (None: the first M), the first
        count[u] of each (None: M; without slots what there is).  Rows behind the
        count are zero."""
        U = self.seqs * self.heads
        k = torch.zeros(U, M, self.d, dtype=torch.bfloat16, device=self.device)
        v = torch.zeros_like(k)
        K_.kvc_page_read(self.pages, slots, count, k, v, self.ws, M=M)
        return k, v

    def hand_over(self, st: DecodeState, slots, count):
        """The budgeted cache st of the same units takes count[u] (int32 [U]) of the
        slots listed in slots[u] (int32 [U][M], M <= cap): rows, positions and
        lengths; utilities and moments start anew, as in load_prefill.  A unit
        whose count or slots are refused (status()) is empty."""
        if st.U != self.seqs * self.heads or slots.shape[1] > st.cap:
            raise ValueError(f"{slots.shape[1]} slots of {self.seqs * self.heads} units for a cache "
                             f"of {st.U} units of {st.cap}")
        K_.kvc_page_read(self.pages, slots, count, st.K, st.V, self.ws)
        st.pos[:, :slots.shape[1]].copy_(slots)
        if st.votes is not None:
            st.votes.fill_(1)
        st.util.fill_(float("inf"))
        behind = torch.arange(slots.shape[1], device=slots.device) >= count.unsqueeze(1)
        held = self.len.repeat_interleave(self.heads).unsqueeze(1)
        taken = (((slots >= 0) & (slots < held)) | behind).all(1) & (count >= 0) & (count <= slots.shape[1])
        st.len.copy_(torch.where(taken, count, 0))
        for t in (st.n, st.mu_k, st.mu_v, st.C):
            t.zero_()

    def status(self) -> int:
        """The first error a call recorded and that has not been read yet (0: none)."""
        return K_.kvc_get_device_status(self.ws)

"""Python binding of include/kda_pages.h: the pages of a paged key-value cache,
handed out to the rows of a page table, taken back, shared and moved, all on the
device and in the order of the stream.

The state is three int32 tensors of the caller's: page_table [N, max_pages] (as
for ``paged_append``; starts as -1), held [N] (pages that each row holds; starts
as 0) and refs [P] (holders of each page; starts as 0, and a page is free where
it is 0; a negative count, of a page of the caller's own, stays what it is).  Checks,
streams and errors are as in ``layers``.
"""
from __future__ import annotations

from array import array
from operator import attrgetter

import torch

from .kda import _empty, _record
from .layers import _call, _cuda, _dense, _dims, _size, _status

_Tensor, _shape, _nbytes = torch.Tensor, attrgetter("shape"), attrgetter("nbytes")


def _fits(*sizes):
    """The C interface's sizes are 32-bit: a larger one would be cut short on its way."""
    for n in sizes:
        if not 0 <= n < 1 << 31:
            raise ValueError(f"a size of {n} is out of range")


def _state(page_table, held, refs, page_size):
    """Device, rows, columns and pages, and the three pointers."""
    dev = _cuda(page_table, "page_table")
    N, cols = _dims(page_table, "page_table", 2)
    P = _dims(refs, "refs", 1)[0]
    _fits(N, cols, P, page_size)
    return (dev, N, cols, P, _dense(page_table, "page_table", (N, cols), torch.int32, dev),
            _dense(held, "held", (N,), torch.int32, dev), _dense(refs, "refs", (P,), torch.int32, dev))


def _pools(pools, P, dev):
    """The pools' addresses and the bytes of a page in each, as arrays on the host.  (A model's layers have dozens of
    pools: each check runs over all of them at once.)"""
    try:
        plain = (set(map(type, pools)) <= {_Tensor} and set(map(_Tensor.get_device, pools)) <= {dev.index}
                 and {s[0] for s in map(_shape, pools)} <= {P} and all(map(_Tensor.is_contiguous, pools)))
    except IndexError:                                                   # a tensor without axes
        plain = False
    if not plain:
        _check_pools(pools, P, dev)
    return array("Q", map(_Tensor.data_ptr, pools)), array("q", [n // P for n in map(_nbytes, pools)] if P else [0] * len(pools))


def _check_pools(pools, P, dev):
    for i, t in enumerate(pools):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"pools[{i}] must be a torch.Tensor")
        if t.device != dev:
            raise ValueError(f"pools[{i}] is on {t.device}, expected {dev}")
        if t.dim() < 1 or t.shape[0] != P:
            raise ValueError(f"pools[{i}] has shape {tuple(t.shape)}, expected {P} pages")
        if not t.is_contiguous():
            raise ValueError(f"pools[{i}] must be contiguous")


def _workspace(workspace, name, stream, dev, *sizes):
    """The workspace (a new one for None, where one is needed), its pointer and its bytes."""
    if workspace is not None:
        n = _dims(workspace, "workspace", 1)[0]
        return workspace, _dense(workspace, "workspace", (n,), torch.uint8, dev), n
    n = _size(name, dev, *sizes)
    if n == 0:
        return None, None, 0
    workspace = _empty(stream, n, torch.uint8, dev)
    return workspace, workspace.data_ptr(), n


def pages_resize(page_table, held, refs, tokens, page_size, workspace=None, status=None, stream=None):
    """Row i gets or gives back pages so that it holds those of tokens[i] tokens (int32; 0 ends the row, a negative
    number leaves it).  Free pages are handed out lowest first; held[i] says what a row has where they run out."""
    dev, N, cols, P, tp, hp, rp = _state(page_table, held, refs, page_size)
    workspace, wp, size = _workspace(workspace, "kda_pages_resize_workspace_size", stream, dev, N, cols, P)
    _call("kda_pages_resize", dev, stream, (), tp, N, cols, hp, rp, P, _dense(tokens, "tokens", (N,), torch.int32, dev),
          page_size, wp, size, _status(status, dev))
    if stream is not None:
        _record(stream, page_table, held, refs, tokens, workspace, status)


def pages_fork(pools, page_table, held, refs, lens, src, dst, page_size, workspace=None, status=None, stream=None):
    """Row dst[i] goes on from the tokens of row src[i] (int32; negative: padding): it shares that row's full pages, and
    a partly filled last page is copied to a free one in every tensor [P, ...] of `pools`.  lens [N] int32: tokens of
    each row; lens[dst[i]] becomes lens[src[i]].  A destination holds no pages before, and is no other pair's row."""
    dev, N, cols, P, tp, hp, rp = _state(page_table, held, refs, page_size)
    F = _dims(src, "src", 1)[0]
    ptrs, sizes = _pools(pools, P, dev)
    workspace, wp, size = _workspace(workspace, "kda_pages_fork_workspace_size", stream, dev, N, cols, F)
    _call("kda_pages_fork", dev, stream, (), ptrs.buffer_info()[0], sizes.buffer_info()[0], len(pools), tp, N, cols, hp, rp, P,
          _dense(lens, "lens", (N,), torch.int32, dev), _dense(src, "src", (F,), torch.int32, dev),
          _dense(dst, "dst", (F,), torch.int32, dev), F, page_size, wp, size, _status(status, dev))
    if stream is not None:
        _record(stream, *pools, page_table, held, refs, lens, src, dst, workspace, status)


def pages_compact(pools, page_table, refs, page_map=None, live=None, workspace=None, status=None, stream=None):
    """Moves the pages in use (refs not 0) to the lowest ids in every tensor [P, ...] of `pools`, and the table (or None) and the
    counts with them.  Returns (page_map [P] int32: each page's new id, -1 for a free one; live [1] int32: pages in use)."""
    dev = _cuda(refs, "refs")
    P = _dims(refs, "refs", 1)[0]
    N, cols = (0, 0) if page_table is None else _dims(page_table, "page_table", 2)
    _fits(N, cols, P)
    ptrs, sizes = _pools(pools, P, dev)
    new = []
    if page_map is None:
        page_map = _empty(stream, (P,), torch.int32, dev)
        mp = page_map.data_ptr()
        new.append(page_map)
    else:
        mp = _dense(page_map, "page_map", (P,), torch.int32, dev)
    if live is None:
        live = _empty(stream, (1,), torch.int32, dev)
        lp = live.data_ptr()
        new.append(live)
    else:
        lp = _dense(live, "live", (1,), torch.int32, dev)
    workspace, wp, size = _workspace(workspace, "kda_pages_compact_workspace_size", stream, dev, P)
    _call("kda_pages_compact", dev, stream, new, ptrs.buffer_info()[0], sizes.buffer_info()[0], len(pools),
          _dense(page_table, "page_table", (N, cols), torch.int32, dev), N, cols,
          _dense(refs, "refs", (P,), torch.int32, dev), P, mp, lp, wp, size, _status(status, dev))
    if stream is not None:
        _record(stream, *pools, page_table, refs, page_map, live, workspace, status)
    return page_map, live

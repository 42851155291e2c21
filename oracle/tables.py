"""Block tables from the requests' lengths, the free list and the slots of ragged tokens.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``).

The tables are those of ``oracle/paged.py`` ([P2] section "输入准备:prepare_for_draft": a slot pool reached through a
table per request).  Pages are handed out one by one, in the requests' order and then the pages', from the end of the free
list; a request is served whole or not at all, and once one that needs pages is not served no later one is.
"""
from __future__ import annotations

import numpy as np

ROW_RANGE, INDEX_RANGE, WRITE_RANGE, NO_PAGES = 8, 1, 2, 32


def n_pages(tokens: int, page_size: int) -> int:
    return -(-tokens // page_size)


def grow(table, page_size, new_len, free_pages, n_free, old_len=None):
    """-> (table, lengths, n_free, status); old_len None: built anew."""
    B, width = table.shape
    out = np.full_like(table, -1) if old_len is None else table.copy()
    lengths = np.zeros(B, np.int64)
    status = 0
    left = int(n_free)
    if not 0 <= left <= len(free_pages):
        status |= ROW_RANGE
        left = min(max(left, 0), len(free_pages))
    wanted, top = 0, left          # pages wanted so far, served or not
    for b in range(B):
        old = 0 if old_len is None else int(old_len[b])
        new = int(new_len[b])
        lengths[b] = old
        if old < 0 or new < 0 or max(old, new) > width * page_size:
            status |= ROW_RANGE
            continue
        first, last = n_pages(old, page_size), n_pages(new, page_size)
        need = max(0, last - first)
        wanted += need
        if need and wanted > top:
            status |= NO_PAGES
            out[b, first:last] = -1
            continue
        lengths[b] = max(old, new)      # a shorter request keeps its pages
        for p in range(first, first + need):
            left -= 1
            out[b, p] = free_pages[left]
            if free_pages[left] < 0:
                status |= INDEX_RANGE
    return out, lengths, left, status


def release(table, page_size, old_len, free_pages, n_free, keep_len=None):
    """-> (table, free_pages, n_free, status)."""
    B, width = table.shape
    out, free = table.copy(), free_pages.copy()
    if not 0 <= n_free <= len(free):
        return out, free, n_free, ROW_RANGE
    status, at, full = 0, int(n_free), False
    for b in range(B):
        old, keep = int(old_len[b]), 0 if keep_len is None else int(keep_len[b])
        if old < 0 or keep < 0 or old > width * page_size:
            status |= ROW_RANGE
            continue
        entries = [p for p in range(n_pages(keep, page_size), n_pages(old, page_size)) if out[b, p] >= 0]
        full = full or at + len(entries) > len(free)
        if full:
            # later requests are counted behind this one, so one without pages alone still "fits"
            status |= WRITE_RANGE
            continue
        for p in entries:
            free[at] = out[b, p]
            out[b, p] = -1
            at += 1
    return out, free, at, status


def slot_map(table, page_size, offsets, lengths, T):
    """-> (slots [T], positions [T], written [T] truth values, status) of the ragged tokens."""
    slots, positions = np.zeros(T, np.int64), np.zeros(T, np.int64)
    written = np.zeros(T, bool)
    status = ROW_RANGE if offsets[-1] > T else 0
    for b in range(len(offsets) - 1):
        lo, hi = int(offsets[b]), int(offsets[b + 1])
        for t in range(lo, min(hi, T)):
            pos = int(lengths[b]) - (hi - t)
            page = table[b, pos // page_size] if 0 <= pos and pos // page_size < table.shape[1] else -1
            slots[t] = -1 if page < 0 else int(page) * page_size + pos % page_size
            positions[t], written[t] = pos, True
            status |= ROW_RANGE if page < 0 else 0
    return slots, positions, written, status

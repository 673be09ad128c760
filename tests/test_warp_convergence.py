"""Warp-wide instructions stand where the warp is whole.

The ``.aligned`` forms (TMEM loads, allocation and release, cluster and named
barriers, register shares) need all 32 lanes of a warp at once.  A branch that
depends on the lane parts them, and only a warp-wide call is sure to join them
again: what the compiler happens to do is no promise.  The kernels' sources are
read here block by block, loops twice, and an aligned instruction that can be
reached with the lanes parted is a failure.
"""

import os
import re

import pytest

from factored_weight_norm_b200 import build as build_mod

ALIGNED = re.compile(r"\b(tmem_ld\d+|tmem_alloc\w*|tmem_dealloc\w*|tmem_relinquish\w*|cluster_sync_all|regs_give|regs_take)\b|bar\.sync")
# calls that every lane has to reach, so that they join the warp
JOINS = re.compile(r"__sync\w+\(\s*\)|__syncthreads_and\(|__syncwarp\(|_sync\(0xffffffffu?\b|\b(mbar_wait_warp|epi_sync|quad_transpose)\(", re.I)
LANE = re.compile(r"\b(lane|threadIdx|row_ok|row|t_ok|et|gl|my_row)\b")
# device functions whose loops end at different times for the lanes of a warp
PARTS = re.compile(r"\bslice_join<")


def _blocks(text):
    """The statements and blocks of C++ source: strings, or (header, [items])."""
    text = re.sub(r"//[^\n]*", "", re.sub(r"/\*.*?\*/", "", text, flags=re.S))
    text = re.sub(r"^\s*#[^\n]*", "", text, flags=re.M)
    text = re.sub(r'"[^"\n]*"', lambda m: re.sub(r"[;{}()]", " ", m[0]), text)
    stack, items, cur, depth = [], [], "", 0
    for ch in text:
        if ch == "{":
            stack.append((items, cur, depth))
            items, cur, depth = [], "", 0
        elif ch == "}":
            if cur.strip():
                items.append(cur.strip())
            inner, (items, head, depth) = items, stack.pop()
            if depth == 0:
                items.append((head.strip(), inner))
                cur = ""
            else:  # braces within an expression: an initialiser
                cur = head
        elif ch == ";" and depth == 0:
            if cur.strip():
                items.append(cur.strip())
            cur = ""
        else:
            depth += (ch == "(") - (ch == ")")
            cur += ch
    assert not stack
    return items


def _condition(head):
    m = re.match(r"(?:else\s+)?(?:if|for|while)\s*(?:constexpr\s*)?\(", head)
    if not m:
        return None
    depth, i = 1, m.end()
    while depth:
        depth += (head[i] == "(") - (head[i] == ")")
        i += 1
    return head[m.end():i - 1]


WHOLE, FIRST, ANY = 0, 1, 2  # which warps may be parted: none, warp 0, any


def _walk(items, parted, found, left):
    """The state behind the items; ``left`` collects the states at which a loop is left or begun again."""
    entry = parted
    for item in items:
        head, inner = item if isinstance(item, tuple) else (item, None)
        cond = _condition(head)
        joins = bool(JOINS.search(head if inner is None else cond or ""))
        parts = WHOLE
        if cond is not None and LANE.search(cond) and not JOINS.search(cond):
            parts = FIRST if re.search(r"warp == 0 && lane == 0|threadIdx\.x == 0$", cond.strip()) else ANY
        chained = re.match(r"else\b", head)
        if not chained:
            entry = parted
        if cond is not None and entry == FIRST and re.search(r"\bwarp (==|>=) [1-9]", cond):
            state = WHOLE
        else:
            state = max(entry, parts)
        if inner is not None:
            if joins:
                entry = parted = state = WHOLE
            loop = re.match(r"(for|while|do)\b", head)
            ends = []
            for _ in range(2 if loop else 1):
                state = max([_walk(inner, state, found, ends if loop else left), *ends])
            if not loop and inner and isinstance(inner[-1], str) and re.match(r"(break|continue|return)\b", inner[-1]):
                left.append(state)
                state = WHOLE
            parted = max(state, parts, parted if chained else entry)
            continue
        if ALIGNED.search(head) and state:
            found.append(" ".join(head.split())[:100])
        if joins:
            parted = WHOLE
        parted = max(parted, parts, ANY if PARTS.search(head) else WHOLE)
    return parted


def _kernels(items):
    for item in items:
        if isinstance(item, tuple):
            if re.match(r"(namespace\b|extern\b)", item[0]) or not item[0]:
                yield from _kernels(item[1])
            elif re.search(r"__(global|device)__", item[0]):
                yield item


def parted_uses(text):
    out = []
    for head, inner in _kernels(_blocks(text)):
        found = []
        _walk(inner, WHOLE, found, [])
        name = re.findall(r"(\w+)\s*\(", re.sub(r"__launch_bounds__\([^)]*\)", "", head))
        out += [f"{name[0] if name else head}: {f}" for f in dict.fromkeys(found)]
    return out


def test_the_reader_sees_parted_warps():
    kernel = "__global__ void k(int n) { %s }"
    for body, ok in (("if (lane == 0) f(); tmem_ld16(a, b);", False),
                     ("if (lane == 0) f(); __syncwarp(); tmem_ld16(a, b);", True),
                     ("if (lane == 0) { f(); } else { g(); } cluster_sync_all();", False),
                     ("if (warp == 1) { if (lane == 0) f(); } else { g(); } tc(); cluster_sync_all();", False),
                     ("if (warp == 1) { if (lane == 0) f(); __syncwarp(); } else { tmem_ld32(a, b); }", True),
                     ("if (warp == 0 && lane == 0) f(); if (warp == 1) { tmem_alloc(a, b); }", True),
                     ("if (!mbar_wait_warp(a, b)) { if (lane == 0) f(); return; } tmem_ld32(a, b);", True),
                     ("for (;;) { tmem_ld32(a, b); if (x) { if (lane == 0) f(); continue; } __syncwarp(); }", False),
                     ("for (int i = 0; i < n; ++i) { tmem_ld32(a, b); if (row_ok) g(); }", False),
                     ("for (int i = 0; i < n; ++i) { tmem_ld32(a, b); if (row_ok) g(); __syncwarp(); }", True),
                     ('if (lane == 0) f(); asm volatile("bar.sync %0, %1;" ::"r"(a), "r"(b) : "memory");', False)):
        assert (not parted_uses(kernel % body)) is ok, body


FILES = ("compose.cuh", "quant8.cuh", "ckpt8.cuh", "linear_tc.cuh", "linear_i8.cuh", "linear_ckpt8.cuh", "linear_slice.cuh")


@pytest.mark.parametrize("name", FILES)
def test_aligned_instructions_meet_whole_warps(name):
    with open(os.path.join(build_mod.CSRC, name)) as f:
        assert not parted_uses(f.read())

"""Bounded waits whose answer steers a warp, read from the kernels' sources (no GPU).

A bounded wait can end differently for the lanes of a warp: each reads the abort flag, the barrier and
the clock for itself.  Code behind it that takes the warp whole (matrix products, shuffles, full-mask
barriers) needs one answer, so outside the helper functions a per-lane wait stands under __all_sync, or
in one lane alone whose answer is shuffled to the others, or nothing goes by its answer ("(void)")."""
import os
import re

import pytest

from paged_attention_relative_gqa_gb300 import build

RINGS = ["decode_masked.cu", "decode.cu"]
VOTED = ["decode_masked.cu", "decode.cu", "prefill_tc.cu", "kv_conv.cu", "prefill_pair.cu", "prefill_masked.cu"]


def code(name):
    with open(os.path.join(build.CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def functions(src):
    """(name, body) of the inline device functions, and what is left of the source without them."""
    found, rest, at = [], "", 0
    for m in re.finditer(r"__device__\s+(?:__forceinline__|__noinline__)\s+[\w:]+\s+(\w+)\([^)]*\)\s*\{", src):
        if m.start() < at:
            continue
        depth, end = 1, m.end()
        while depth:
            depth += {"{": 1, "}": -1}.get(src[end], 0)
            end += 1
        found.append((m.group(1), src[m.end():end - 1]))
        rest += src[at:m.start()]
        at = end
    return found, rest + src[at:]


def lone_waits(src):
    """Statements outside the helpers that wait by lane: neither voted on (at once, or by way of a variable), nor
    made by lane 0 alone, nor with an answer that is thrown away or only masks the lane's own keys."""
    helpers, rest = functions(src)
    by_lane = {"mbar_wait_limit"}
    for name, body in helpers:
        if "__all_sync" not in body and any(w + "(" in body for w in by_lane):
            by_lane.add(name)
    call = re.compile(r"\b(?:%s)\(" % "|".join(sorted(by_lane)))
    found = []
    for m in re.finditer(r"[^;{}]+", rest):
        s = m.group().strip()
        if not call.search(s) or re.search(r"__all_sync|lane == 0|\(void\)", s):
            continue
        if re.search(r"if \(lane == 0\) \{\s*$", rest[:m.start()]):
            continue
        kept = re.search(r"(\w+) = [^=]*\b%s" % call.pattern, s)
        after = rest[m.end():m.end() + 2500]
        if kept and re.search(r"\b%s = __all_sync\(0xffffffffu,\s*%s\b" % (kept.group(1), kept.group(1)), after):
            continue
        uses = re.findall(r"[^;{}]*\bok\b[^;{}]*", after.split("for (")[0]) if kept and kept.group(1) == "ok" else []
        if uses and all(u.strip() == "if (!ok) bad = ~0ull" for u in uses):
            continue
        found.append(s)
    return found


def test_the_reader_of_sources():
    helper = "__device__ __forceinline__ bool w(int* p) { if (*p) { return mbar_wait_limit(p); } return true; }"
    voted = helper.replace("return true", "return __all_sync(~0u, *p)")
    assert lone_waits(helper + "void k() { const bool ok = w(p); }") == ["const bool ok = w(p)"]
    assert lone_waits(helper + "void k() { ok = __all_sync(~0u, w(p)); if (lane == 0) ok = w(p); }") == []
    assert lone_waits(helper + "void k() { ok = w(p); ok = __all_sync(0xffffffffu, ok && w(q)); if (!ok) return; }") == []
    assert lone_waits(helper + "void k() { ok = w(p); if (!ok) bad = ~0ull; }") == []
    assert lone_waits(helper + "void k() { ok = w(p); if (!ok) bad = ~0ull; if (ok) f(); }") == ["ok = w(p)"]
    assert lone_waits(voted + "void k() { ok = w(p); if (n) ok = mbar_wait_limit(p); }") == ["if (n) ok = mbar_wait_limit(p)"]


@pytest.mark.parametrize("name", VOTED)
def test_waits_of_a_warp_have_one_answer(name):
    assert lone_waits(code(name)) == []


@pytest.mark.parametrize("name", RINGS)
def test_a_stage_is_handed_back_only_after_a_wait_that_succeeded(name):
    """The wait for a tile is followed at once by the way out, before any arrival that frees its stage, and the
    loader looks at the abort flag again after a stage or a Q slot has come back."""
    src = code(name)
    waits = [m for m in re.finditer(r"const bool ok = [^;]*&full\[[^;]*;", src)]
    assert len(waits) == 1
    assert re.match(r"\s*if \(!ok\) \{[^{}]*break;\s*\}", src[waits[0].end():])
    frees = [s for s in re.split(r"[;{}]", src) if re.search(r"wait\w*\(&q?empty", s)]
    assert len(frees) == 2 and all("&& !*abort_flag" in s for s in frees)


def test_the_prefill_fills_no_slot_again_whose_wait_failed():
    """Its warps go on after a timeout.  A V slot goes back with the product that read it; the bias loader looks at
    the flag again."""
    src = code("prefill_tc.cu")
    assert src.count("umma_commit_warp(&v_empty") == 1
    assert re.search(r"if \(pv_ok\) \{(?:(?!\n          \}).)*umma_commit_warp\(&v_empty\[vs\]\);", src, re.S)
    assert re.search(r"wait_flag\(&b_empty\[slot\][^;]*&&\s*!\*abort_flag\)", src)

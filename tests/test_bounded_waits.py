"""Waits of the kernels that run warp-wide instructions, read in their sources.

A bounded wait may give up, and its lanes may do so one by one.  Code of a whole
warp that goes on to votes, shuffles or tcgen05 loads needs one answer for all
lanes, or the lanes that go on wait for the others for good: no run shows that
unless a wait runs out, so it is read off the source.
"""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "rag_precomputed_kv_gb300", "csrc")
ROLE = re.compile(r"^    (?:\} else )?if \((?:kV && )?warp (==|<|>=) (\d+)\) \{|^    \} else \{", re.M)


def _source(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def _roles(text):
    """(condition, text) of each warp role of the file's kernels."""
    m = list(ROLE.finditer(text))
    return [((a.group(1), a.group(2)), text[a.end():b.start() if b else len(text)]) for a, b in zip(m, m[1:] + [None])]


PLAIN = re.compile(r"\bmbar_wait(?:_cluster)?\(")


def test_attention_roles_leave_together():
    """k_attention_tc: a lane that lost a wait takes part in its warp's votes and
    leaves at one of them with the others, never before."""
    roles = dict(reversed(_roles(_source("kvr_attention_tc.cu"))))   # (the first of each condition)
    for cond in (("<", "8"), ("==", "9"), (">=", "10")):
        text = roles[cond]
        item = text[text.index("for (int it = blockIdx.x; it < n_items; it"):]
        # every item starts with a vote that knows of the waits before it
        assert re.match(r"for \([^)]*\) \{\s*(int [^;]*;\s*bool [^;]*;\s*int64_t [^;]*;\s*\{\s*)?"
                        r"const Geo \*gp = geo_wait\(gk, ok\);\s*if \(!gp\)", item), item[:300]
        if cond != ("==", "9"):   # (no lane of the MMA warp needs another within an item)
            for m in PLAIN.finditer(item):
                line = item[item.rindex("\n", 0, m.start()):item.index("\n", m.end())]
                after = item[item.index("\n", m.end()):][:120]
                assert "__all_sync(" in line or "ok = mbar_wait(" in line or re.match(r"\s*ok = false;\s*\*abort_flag = 1;\s*\}", after), line
    softmax = roles["<", "8"]
    assert "__any_sync(0xffffffffu, corr != 1.f || !ok)" in softmax and "if (__any_sync(0xffffffffu, !ok))" in softmax
    body = roles["==", "9"][roles["==", "9"].index("geo_done(gk)") + 12:]
    assert not re.search(r"(?<!mbar)_sync\(|__syncwarp|tmem_(ld|st)", body)


def test_decode_warps_wait_with_one_answer():
    """k_decode_attention: a tile's wait is voted on, thread 0's wait for a free
    stage with the next tile's."""
    text = _source("kvr_decode.cu")
    loop = text[text.index("for (int j = 0; j < n_t; ++j) {"):text.index("if (!ok)\n        *cta_err = 1;")]
    waits = [loop[loop.rindex("\n", 0, m.start()):m.end()] for m in re.finditer(r"\bdec_wait\(", loop)]
    assert len(waits) == 2 and "__all_sync(0xffffffffu, ok && " in waits[0] and "ok = dec_wait(" in waits[1]
    assert loop.count("break;") == 1


def test_key_weight_warps_read_the_abort_flag_with_one_answer():
    """Both tensor-core kernels: lanes that go on to tcgen05 loads agree on whether
    the CTA gave up (a vote, or one thread's reading of it)."""
    text = _source("kvr_key_weights_tc.cu")
    reads = [m.group(0).strip() for m in re.finditer(r"[^\n]*\*abort_(?:flag|seen)\b[^\n]*", text[text.index("template <int NC>\n__global__"):])]
    reads = [r for r in reads if not r.startswith("volatile int")]
    assert reads == ["*abort_flag = 0;", "if (__any_sync(0xffffffffu, *abort_flag != 0))", "*abort_flag = *abort_seen = 0;",
                     "*abort_seen = *abort_flag;", "if (*abort_seen) {"]


def test_shared_prefix_kernels_read_what_they_may():
    """A programmatic launch promises what earlier kernels wrote to a grid that
    waited itself.  A role of the shared-prefix kernels that reads ahead of its wait
    has first seen that an earlier grid passed its own wait on."""
    text = _source("kvr_shared_tc.cu")
    roles = dict(reversed(_roles(text)))
    wait, flat = "pdl_wait_prerequisites();", lambda s: re.sub(r"\s+", " ", s)
    softmax, load, mma = (flat(roles[c]) for c in (("<", "8"), ("==", "8"), ("==", "9")))
    for role in (softmax, mma):
        before = role.split(wait, 1)[0]
        assert "seg(" not in before and "mbar_wait" not in before and "tmem_" not in before
    seen = "waited = !relay_seen(a.relay, a.call); if (waited) " + wait
    assert seen in load and not re.search(r"seg\(|tma_load_2d\(", load[:load.index(seen)])
    assert softmax.index(wait) < softmax.index("relay_store(a.relay + 1, a.call);") < softmax.index("pdl_launch_dependents();")

    def kernel(name):
        start = text.index("    " + name)
        return flat(text[start:text.index("\n}\n", start)])
    own = kernel("k_shared_own_decode(")
    seen = "waited = lane == 0 && !relay_seen(pa.relay + 1, pa.call); waited = __shfl_sync(0xffffffffu, waited, 0); } if (waited) " + wait
    assert seen in own and not re.search(r"reqs\[|load_piece\(\);|issue\(\);|load_queries\(it", own[:own.index(seen)])
    prologue = kernel("k_shared_prologue(")
    assert prologue.index(wait) < prologue.index("relay_store(a.relay, a.call);") < prologue.index("pdl_launch_dependents();")
    assert not re.search(r"reqs\[", prologue[:prologue.index(wait)])


def test_eviction_kernels_read_uploaded_tables_behind_their_own_wait():
    text = _source("kvr_evict.cu")
    for name in ("k_evict_select(", "k_evict_move(", "k_evict_unit("):
        start = text.index("    " + name + "const __grid_constant__")
        body = text[start:text.index("\n}\n", start)]
        before = re.split(r"(?:if \(a\.reqs\)\s*)?pdl_wait_prerequisites\(\);", body, maxsplit=1)
        assert len(before) == 2 and not re.search(r"reqs\)?\[", before[0]), name

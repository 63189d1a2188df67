"""Waits that are given up: what the sources have to keep to, so that threads which meet at barriers and in shuffles give up
together or not at all (a thread that leaves alone holds the others up for good).  Read from the sources: no GPU is used, and
none is made to wait."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "llama_decoder_block_fwd_gb300", "csrc")


def _code(name):
    text = open(os.path.join(CSRC, name)).read()
    return re.sub(r"//[^\n]*", "", text), text


def test_softmax_threads_of_the_8_bit_paged_attention_never_leave_alone():
    """Their loop runs over the range's tiles, whatever a wait says: no wait's result decides on anything."""
    _, text = _code("decode_attn8p.cu")
    role = text[text.index("- softmax warps"):text.index("// Joins the parts")]
    role = re.sub(r"//[^\n]*", "", role)
    assert role.count("softmax_sync_dp(") == 2 and "warp_max_dp(" in role       # (what they meet in is there)
    assert not re.search(r"\bbreak\b|\bgoto\b|\bok\b", role)
    assert not re.search(r"(if|while|&&|\|\||=|return)\s*\(?\s*!?\s*(wait_for|mbar_wait)", role)


def test_loading_warp_of_the_8_bit_paged_attention_gives_up_as_one():
    """Its lanes convert q together, so each lane's waits there are put to a vote before the shuffles."""
    code, _ = _code("decode_attn8p.cu")
    put_q = code[code.index("auto put_q"):code.index("int it = 0;")]
    waits = put_q.index("wait_for("), put_q.rindex("wait_for(")
    assert "return false" not in put_q[:waits[1]] and put_q.index("__all_sync(0xffffffffu, free)") > waits[1]
    assert put_q.index("__shfl_xor_sync") > put_q.index("__all_sync")


def test_takers_of_beam_selection_give_up_together():
    """They meet at one_gave_up alone, which gives all of them the same answer; a wait is a whole warp's, and one that runs out goes
    there too; whatever meets ends its caller where it fails; and every warp meets the others once more at its end."""
    code, _ = _code("beam.cu")
    part = code[code.index("auto meet ="):code.index("constexpr int BM_MOST")]
    assert not re.search(r"bar\.sync|barrier\.cta|__syncthreads", part)
    waits = list(re.finditer(r"if \(!__all_sync\(0xffffffffu, mbar_wait\([^;]*\) return give_up\(\);", part))
    assert len(waits) == part.count("mbar_wait(") == 2
    for call in re.finditer(r"\b(meet|count|squeeze|cut|settle|take)\(", part[:part.rindex("meet();")]):
        before = part[max(0, call.start() - 40):call.start()].rstrip()
        assert re.search(r"(!|return)$", before), part[call.start() - 40:call.end() + 20]
    assert re.search(r"meet\(\);\s*\}\s*$", part)
    common, _ = _code("common.cuh")
    assert "barrier.cta.red.or.pred" in common


def test_join_of_beam_selection_looks_for_no_list_where_none_is():
    """After a first kernel that gave up, a row's record of its lists may be whatever the workspace held: it is held against the
    lists that there are, and a request's against the room for them, before anything is indexed by it."""
    code, _ = _code("beam.cu")
    join = code[code.index("beam_merge_kernel("):code.index("int64_t select_grid(")]
    checks = join.index("(int64_t)pieces.slot + pieces.n <= p.n_lists"), join.index("<= BM_LISTS")
    assert "pieces.slot >= 0 && pieces.n >= 0" in join and max(checks) < join.index("row_of[l]") and max(checks) < join.index("p.keys[")

"""What the attention kernel's source has to keep and no run can show (no GPU needed)."""
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCE = os.path.join(ROOT, "speculative_decoding_drafter_gb300", "csrc", "attention.cu")


def register_splits(text):
    """The calls that change a warpgroup's registers, each with the heads of the blocks that it stands in."""
    text = re.sub(r"//[^\n]*", "", text)
    text = text[text.index("attention_kernel("):text.index("combine_kernel(")]
    calls, heads, head = [], [], ""
    at = 0
    while at < len(text):
        c = text[at]
        call = re.match(r"reg_(?:dec|inc)<", text[at:])
        if call:
            calls.append(list(heads))
        if c == "{":
            heads.append(" ".join(head.split()))
            head = ""
        elif c == "}":
            heads.pop()
            head = ""
        elif c == ";":
            head = ""
        else:
            head += c
        at += 1
    return calls


def shared_by_a_warpgroup(heads):
    """Whether the conditions on `warp` hold for all four warps of a warpgroup or for none."""
    return all(re.fullmatch(r"(else )?if \(warp < 4( \+ 4 \* QT)?\)", h) for h in heads if re.search(r"\bwarp\b", h))


def test_a_warpgroup_changes_its_registers_in_one_place():
    """setmaxnreg is one instruction for the four warps of a warpgroup: two of them in the branches of its roles are
    undefined, and what waits for the registers waits without a limit."""
    calls = register_splits(open(SOURCE).read())
    assert len(calls) == 3  # control, softmax, widening
    assert all(shared_by_a_warpgroup(heads) for heads in calls)
    assert len({tuple(h) for h in calls}) == len(calls)


def test_the_check_sees_a_split_by_roles():
    text = """attention_kernel(int a) { if (warp == 0 || warp == 3) { if constexpr (S) reg_dec<1>(); }
              else if (warp < 4) { reg_dec<1>(); } } combine_kernel("""
    calls = register_splits(text)
    assert [shared_by_a_warpgroup(h) for h in calls] == [False, True]

"""Warps that meet at a barrier of their group leave their loop together: a warp that left by itself, because a wait of its own
ran out, would leave the others at the barrier for ever."""
import pathlib
import re

SOURCE = pathlib.Path(__file__).resolve().parent.parent / "mla_latent_cache_attention_gb300" / "csrc" / "mla_fp4.cuh"


def test_the_loaders_of_the_4_bit_decode_leave_together():
    """A loader warp whose wait runs out goes on to the barrier of the next item (next_item), which hears of it and ends all of them."""
    text = SOURCE.read_text()
    head, end = "for (int gt = 0; ok && have; ++gt) {", "errbits = __reduce_or_sync"
    assert text.count(head) == 1
    body = text[text.index(head):text.index(end)]
    loop, left = body.rsplit("have2 = c.table != nullptr;", 1)
    # the loop is left early by `mine` alone ...
    assert re.findall(r"\bcontinue\b|\bok\s*=|\breturn;", loop) == []
    assert loop.count("break;") == len(re.findall(r"if \(!\(mine = [^;]*\)\) break;|if \(!mine\) break;", loop)) > 0
    # ... and then the cursor goes on to the barrier
    assert re.fullmatch(r"\s*}\s*if \(!mine\)\s*while \(c\.table\) advance\(c\);\s*", left)
    item = text[text.index("auto next_item = "):text.index("auto advance = ")]
    assert re.search(r"if \(!group_wait\(.*, mine\)\) {\s*ok = false;\s*c\.table = nullptr;", item)

"""Rules of the 8-bit attention's source that no run can show without a failing
GPU: they are read from the text."""
import re

from tests.test_latent_rules import source


def softmax_role():
    """The softmax role's loop over the pieces."""
    text = source("qlatent_attend.cu")
    role = text[text.index("else if (warp >= 4)"):text.index("if (kCl > 1 && it == 0")]
    return role[role.index("while (more)"):]


def test_softmax_threads_leave_together():
    """The role's named barriers count every softmax thread.  A bounded wait may run out in some of them alone, so a
    thread leaves a loop with such a barrier only where all of them vote (named_any), behind such a vote (ok is then
    false in all of them), or where none is missing: at the end of a cluster's only piece."""
    role = softmax_role()
    ends = r"if \(named_any<1, kSoftThreads>\(!ok\)\) \{ ok = false; break; \}"
    assert len(re.findall(ends, role)) == 2
    assert len(re.findall(r"if \(again \|\| !named_any<1, kSoftThreads>\(grow \|\| !ok\)\) break;", role)) == 1
    # out of the tile loop directly behind the inner loop, whose ends are the votes above
    inner = role[role.index("for (;; again = true)"):]
    after = inner[re.search(ends, inner).end():]
    assert after.index("if (!ok) break;") < after.index("mbar_arrive") and role.count("if (!ok) break;") == 1
    assert not re.search(r"\bok = [^;]*wait", after[:after.index("if (!ok) break;")])
    left = re.sub(ends, "", role)
    left = left.replace("if (again || !named_any<1, kSoftThreads>(grow || !ok)) break;", "").replace("if (!ok) break;", "")
    assert [m.group(1).strip() for m in re.finditer(r"([^;{}]*)\bbreak;", left)] == [""]      # the cluster's
    left = re.sub(r"\{ return [^{};]*; \}", "", left)          # (lambdas)
    assert not re.search(r"\breturn\b|\bgoto\b", left)


def test_no_wait_is_unbounded():
    """A wait is one try, then mbar_wait, which counts its tries: nothing polls on its own."""
    for name in ("qlatent_attend.cu", "pages.cu", "qlatent_append.cu"):
        text = source(name)
        assert not re.search(r"mbarrier\.(try|test)_wait|while \((true|1)\)|while \(![a-z_:]*wait", text), name
    text = source("qlatent_attend.cu")
    assert len(re.findall(r"\bmbar_try_wait\(", text)) == 1 and len(re.findall(r"\bmbar_wait\(", text)) == 1
    assert text.count("for (;;") == 1           # the weights' second forming, which ends where `again` is set
    assert "for (;; again = true)" in text
